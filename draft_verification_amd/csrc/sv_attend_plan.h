// How spec_verify_attend shares its work out: plain C++, so that it can be looked
// at without a GPU.
#ifndef SV_ATTEND_PLAN_H
#define SV_ATTEND_PLAN_H

namespace sv {

constexpr int kAttendTokens = 32; // tokens that a wavefront takes at a time
constexpr int kAttendWaves = 4;

struct AttendPlan {
    int tiles;     // of 16 rows (a row and a head of the block each) to a workgroup
    int blocks;    // workgroups for a block's rows
    int splits;    // at most, of a sequence's length
    int span;      // tokens of a split
};

// Most tiles that a workgroup keeps its sums in registers for.
inline int attend_most_tiles(int dim) { return dim > 128 ? 4 : 9; }

// Tiles of the kernel that takes n of them.
inline int attend_tiles(int dim, int n)
{
    if (n <= 3) return n;
    if (dim > 128) return 4;
    return n <= 5 ? 5 : 9;
}

// dim: 64, 128 or 256 (the head's, rounded up).  rows: of all heads that share a
// key-value head.  len: tokens that a sequence may see.
inline AttendPlan attend_plan(long long B, int kv_heads, int dim, long long rows, long long len)
{
    AttendPlan p;
    const long long n = (rows + 15) / 16, most = attend_most_tiles(dim);
    p.blocks = (int)((n + most - 1) / most);
    p.tiles = attend_tiles(dim, (int)((n + p.blocks - 1) / p.blocks));
    const long long step = kAttendTokens * kAttendWaves;
    const long long groups = B * kv_heads * p.blocks;
    long long splits = (2048 + groups - 1) / groups;
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
