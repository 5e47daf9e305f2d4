// Which kernel spec_verify_head takes for a number of rows: plain C++, so that
// the choice can be looked at without a GPU.
#ifndef SV_HEAD_CHOICE_H
#define SV_HEAD_CHOICE_H

namespace sv {

constexpr int kHeadStrip = 64; // vocabulary rows of a strip

// Time of a step of the tiles of 16, 32 and 64 rows, in us, with up to one workgroup
// to each of the 256 compute units and with two (measured at H = 4096, V = 16000 and
// 32000, four blocks of rows).  FP4, INT4 of 32, of 64, of 128.
constexpr float kTileStep[4][3][2] = {
    {{0.57f, 0.92f}, {0.87f, 1.31f}, {1.25f, 2.08f}},
    {{1.09f, 1.50f}, {1.56f, 2.14f}, {2.15f, 3.17f}},
    {{0.83f, 1.25f}, {1.25f, 1.73f}, {1.74f, 2.66f}},
    {{0.84f, 1.24f}, {1.11f, 1.58f}, {1.65f, 2.42f}},
};

// Hidden rows of the tile that a call takes (16, 32, 64), or 0: the split-K
// workgroups of few rows.  group: values to a scale.
inline int head_tile_rows(int rows, long long vocab, bool fp4, int group)
{
    // A tile workgroup does the work of four strips for its rows but takes the
    // same time however few of them there are, while the split-K workgroups, four
    // times as many for every 16 rows, do 1050 steps of a strip and 16 rows a us
    // on the whole chip whatever their number.  So what is quickest depends on how
    // many tiles there are, and the times above say it.  us as split-K and as tiles
    // of 16, 32 and 64, H = 4096:
    //   FP4   16 rows of V = 16000   10   19   24   30
    //         100 of 8000            30   17   24   31
    //         128 of 16000           62   27   28   34
    //         256 of 32000          243  101   73   66
    //   INT4  100 of 8000, group 64  30   25   33   46
    //         128 of 16000           61   38   38   50
    //         256 of 32000          241  134  105   85
    // Where the weights' bytes bound both they come close, and the times above say
    // nothing of bytes (75 us is 1.34 a step, for 0.92), so up to 8 rows it is split-K.
    // us as split-K and as tiles of 16, V = 129280:
    //   rows                  4         8         9        16        17
    //   FP4, H = 4096      45  51    47  51    47  51    57  52    98  63
    //   FP4, H = 7168      75  75    78  75    80  75    98  75   170 104
    //   INT4 of 32, 4096   53  58    54  57    54  57    61  58   107  82
    //   INT4 of 128, 7168  76  78    78  76    80  76    96  77   166 115
    if (rows <= 8) return 0;
    const long long strips = (vocab + kHeadStrip - 1) / kHeadStrip;
    const int kind = fp4 ? 0 : group == 32 ? 1 : group == 64 ? 2 : 3;
    float least = (float)strips * ((rows + 15) / 16) / 1050.0f;
    int best = 0;
    for (int i = 0; i < 3; ++i) {
        const int tile = 16 << i;
        const long long n = (strips + 3) / 4 * ((rows + tile - 1) / tile);
        const float one = kTileStep[kind][i][0], two = kTileStep[kind][i][1];
        const float t = n <= 256 ? one : n <= 512 ? two : two * ((float)n / 512.0f) + one / 2;
        if (t < least) least = t, best = tile;
    }
    return best;
}

// Whether a tile's workgroups read the weights once: there is one block of rows.
// (Tiles of 64 rows make no difference of it.)
constexpr bool head_tile_once(int tile_rows, long long blocks) { return tile_rows < 64 && blocks == 1; }

} // namespace sv

#endif // SV_HEAD_CHOICE_H
