// How spec_verify_attend shares its work out: plain C++, so that it can be looked
// at without a GPU.
#ifndef SV_ATTEND_PLAN_H
#define SV_ATTEND_PLAN_H

namespace sv {

constexpr int kAttendTokens = 32;  // tokens that a wavefront takes at a time
constexpr int kAttendWaves = 4;
constexpr int kAttendUnit = kAttendTokens * kAttendWaves; // tokens by which work is shared out
constexpr int kAttendBegin = 2;    // units that beginning and ending a sequence counts for
constexpr int kAttendBatch = 256;  // most sequences of a launch

struct AttendPlan {
    bool shared;   // the wavefronts share the tokens and split the rows, not the other way round
    int tiles;     // of 16 rows (a row and a head of the block each) to a wavefront
    int rows;      // of a workgroup
    int blocks;    // workgroups for a block's rows
    int shares;    // equal shares of all sequences' tokens, of which each key-value head and block of rows takes all
    int batch;     // sequences of a launch
};

inline long long attend_units(long long tokens) { return (tokens + kAttendUnit - 1) / kAttendUnit; }

// dim: 64, 128 or 256 (the head's, rounded up).  rows: of all heads that share a
// key-value head.  len: tokens that a sequence may see.
inline AttendPlan attend_plan(long long B, int kv_heads, int dim, bool e4m3, long long rows, long long len)
{
    AttendPlan p;
    const long long n = (rows + 15) / 16;
    p.shared = n > (dim > 128 ? 1 : 3);
    if (p.shared) {
        const long long most = kAttendWaves * (dim > 128 ? 1 : 3); // tiles of a workgroup
        p.blocks = (int)((n + most - 1) / most);
        p.tiles = (int)(((n + p.blocks - 1) / p.blocks + kAttendWaves - 1) / kAttendWaves);
    } else {
        p.blocks = 1;
        p.tiles = (int)n;
    }
    p.rows = p.tiles * 16 * (p.shared ? kAttendWaves : 1);
    // as many workgroups as the chip holds at once
    const int at_once = dim == 64 ? 3 : !p.shared && !e4m3 && (dim == 256 || p.tiles == 3) ? 1 : 2;
    const long long each = (long long)kv_heads * p.blocks;
    const long long cost = attend_units(len) + kAttendBegin;
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
