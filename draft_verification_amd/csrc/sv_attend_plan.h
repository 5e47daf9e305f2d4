// How spec_verify_attend shares its work out: plain C++, so that it can be looked
// at without a GPU.
#ifndef SV_ATTEND_PLAN_H
#define SV_ATTEND_PLAN_H

#ifndef SV_TARGET
#define SV_TARGET 2048
#endif
namespace sv {

constexpr int kAttendTokens = 32; // tokens that a wavefront takes at a time
constexpr int kAttendWaves = 4;

struct AttendPlan {
    bool shared;   // the wavefronts share the tokens and split the rows, not the other way round
    int tiles;     // of 16 rows (a row and a head of the block each) to a wavefront
    int rows;      // of a workgroup
    int blocks;    // workgroups for a block's rows
    int splits;    // at most, of a sequence's length
    int span;      // tokens of a split
};

// dim: 64, 128 or 256 (the head's, rounded up).  rows: of all heads that share a
// key-value head.  len: tokens that a sequence may see.
inline AttendPlan attend_plan(long long B, int kv_heads, int dim, long long rows, long long len)
{
    AttendPlan p;
    const long long n = (rows + 15) / 16;
    p.shared = n > (dim > 128 ? 1 : 2);
    if (p.shared) {
        const long long most = kAttendWaves * (dim > 128 ? 1 : 3); // tiles of a workgroup
        p.blocks = (int)((n + most - 1) / most);
        p.tiles = (int)(((n + p.blocks - 1) / p.blocks + kAttendWaves - 1) / kAttendWaves);
    } else {
        p.blocks = 1;
        p.tiles = (int)n;
    }
    p.rows = p.tiles * 16 * (p.shared ? kAttendWaves : 1);
    const long long step = kAttendTokens * kAttendWaves;
    const long long groups = B * kv_heads * p.blocks;
    long long splits = (SV_TARGET + groups - 1) / groups;
    if (splits > (len + step - 1) / step) splits = (len + step - 1) / step;
    if (splits < 1) splits = 1;
    p.span = (int)(((len + splits - 1) / splits + step - 1) / step * step);
    if (p.span < step) p.span = (int)step;
    p.splits = (int)((len + p.span - 1) / p.span);
    if (p.splits < 1) p.splits = 1;
    return p;
}

} // namespace sv

#endif // SV_ATTEND_PLAN_H
