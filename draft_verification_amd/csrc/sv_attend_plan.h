// How spec_verify_attend shares its work out: plain C++, so that it can be looked
// at without a GPU.
#ifndef SV_ATTEND_PLAN_H
#define SV_ATTEND_PLAN_H

namespace sv {

constexpr int kAttendTokens = 32;  // tokens that a wavefront takes at a time
constexpr int kAttendWaves = 4;
constexpr int kAttendUnit = kAttendTokens * kAttendWaves; // tokens by which work is shared out
constexpr int kAttendBatch = 256;  // most sequences of a launch

struct AttendPlan {
    bool shared;   // the wavefronts share the tokens and split the rows, not the other way round
    int tiles;     // of 16 rows (a row and a head of the block each) to a wavefront
    int rows;      // of a workgroup
    int blocks;    // workgroups for a block's rows
    int shares;    // equal shares of all sequences' tokens, of which each key-value head and block of rows takes all
    int begin;     // units that beginning and ending a sequence counts for
    int batch;     // sequences of a launch
};

inline long long attend_units(long long tokens) { return (tokens + kAttendUnit - 1) / kAttendUnit; }

// Workgroups of a compute unit, by the registers that the kernel needs.
constexpr int attend_at_once(int dim, bool e4m3, int tiles, bool shared)
{
    return dim == 64 && tiles <= 1 + e4m3 ? 3 : dim > 128 && !shared && !e4m3 ? 1 : 2;
}

// dim: 64, 128 or 256 (the head's, rounded up).  rows: of all heads that share a
// key-value head.  len: tokens that a sequence may see.
inline AttendPlan attend_plan(long long B, int kv_heads, int dim, bool e4m3, long long rows, long long len)
{
    AttendPlan p;
    const long long n = (rows + 15) / 16;
    // us of 64 sequences of 200 to 8000 tokens and eight key-value heads, split by tokens and by
    // rows: of 64 columns in bf16 one tile of rows 73 and 73, two 96 and 76; in e4m3 two 47 and
    // 53, three 73 and 62; of 128 in bf16 two 129 and 134, three 179 and 141; in e4m3 three 95
    // and 104 (four tiles' sums, or two of 256 columns, do not fit the registers of a wavefront)
    p.shared = n > (dim > 128 ? 1 : dim / 64 + e4m3);
    if (p.shared) {
        const long long most = kAttendWaves * (dim > 128 ? 1 : 3); // tiles of a workgroup
        p.blocks = (int)((n + most - 1) / most);
        p.tiles = (int)(((n + p.blocks - 1) / p.blocks + kAttendWaves - 1) / kAttendWaves);
    } else {
        p.blocks = 1;
        p.tiles = (int)n;
    }
    p.rows = p.tiles * 16 * (p.shared ? kAttendWaves : 1);
    // What a piece of a sequence takes beside its tokens is about that of 256 tokens.  In bf16 with
    // heads of 256 or one tile of rows it is that of 128, and where the sums of three tiles meet at
    // its end (tokens split, which e4m3 of 128 columns alone has) that of 512.  us with 1, 2 and 4
    // units, 64 sequences of 200 to 8000 tokens, eight key-value heads.  Tokens split: bf16, one
    // tile, of 64 columns 64, 64 and 67, of 128 112, 119 and 121, of 256 219, 217 and 241, two of
    // 128 122, 122 and 129; e4m3, of 64 one tile 40, 38 and 40, two 49, 45 and 46, of 128 one 67,
    // 65 and 67, two 81, 79 and 79, three 101, 96 and 90, of 256 one 138, 133 and 138.  Rows split,
    // nine tiles: bf16, of 64 124, 125 and 130, of 128 202, 202 and 207, of 256 604, 620 and 650;
    // e4m3, 121, 119 and 126, 178, 174 and 187, and 570, 584 and 612 (here 2 is not the best).
    // 256 sequences of 500 to 4000, bf16 of 128, nine tiles: 534, 522 and 526
    p.begin = !e4m3 && (dim > 128 || (!p.shared && p.tiles == 1)) ? 1 : !p.shared && p.tiles == 3 ? 4 : 2;
    // As many workgroups as the chip holds at once.  Half as many, and twice: 72 and 64 us for 60,
    // 92 and 72 for 76, 125 and 105 for 99, 817 and 549 for 519
    const int at_once = attend_at_once(dim, e4m3, p.tiles, p.shared);
    const long long each = (long long)kv_heads * p.blocks;
    const long long cost = attend_units(len) + p.begin;
    p.batch = (int)((1ll << 30) / cost < kAttendBatch ? (1ll << 30) / cost : kAttendBatch);
    if (B < p.batch) p.batch = (int)B;
    long long shares = 256 * at_once / each / 8 * 8;
    if (shares < 8) shares = 8;
    const long long most = (p.batch * cost + 7) / 8 * 8;
    p.shares = (int)(shares < most ? shares : most);
    return p;
}

} // namespace sv

#endif // SV_ATTEND_PLAN_H
