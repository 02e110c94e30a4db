// How calls of the log probabilities are cut, for the tests: reads lines of
// "tokens hidden vocab top_k dtype backward live" and prints the layout of each (of a
// forward call: of its first and of its last chunk) as name=value pairs, with the splits
// that the device chooses for dH where `live` rows take part (head_layout.cpp, linked in).
#include <algorithm>
#include <cstdio>

#include "head_layout.h"

using namespace dmuon;

int main() {
    long long t, d, v, live;
    int k, dt, back;
    while (std::scanf("%lld %lld %lld %d %d %d %lld", &t, &d, &v, &k, &dt, &back, &live) == 7) {
        dmuon_head_desc desc{t, d, v, k, dt};
        if (probs_check_desc(&desc, back != 0) != DMUON_OK) {
            std::printf("refused=1\n");
            continue;
        }
        const int64_t chunk = back ? t : std::min<int64_t>(probs_chunk(desc), t);
        const int64_t last = t - (t - 1) / chunk * chunk;
        desc.tokens = chunk;
        const ProbsLayout P = probs_layout_of(desc, back != 0);
        desc.tokens = last;
        const HeadLayout E = probs_layout_of(desc, back != 0).head;
        const HeadLayout& L = P.head;
        const int tiles = (int)(ceil_div(L.hidden, kHeadTile) * ceil_div(live, kHeadTile));
        const int slabs = (int)(round_up(std::min(L.piece, L.vocab), kHeadSlab) / kHeadSlab);
        std::printf("refused=0 chunk=%lld last=%lld keep=%d s_tp=%d s_tq=%d last_s_tp=%d last_s_tq=%d stream=%d last_stream=%d "
                    "pieces=%d piece=%lld low=%d dh_tq=%d splits=%d room=%d live_splits=%d cached=%d dw_cached=%d dw_tp=%d dw_tq=%d dw_splits=%d dh_tp=%d t_pad=%lld\n",
                    (long long)chunk, (long long)last, P.keep_logits, L.s_tile.tp, L.s_tile.tq, E.s_tile.tp, E.s_tile.tq,
                    L.stream_weight, E.stream_weight, L.pieces, (long long)L.piece, L.low, L.dh_tile.tq, L.splits, L.dh_room,
                    L.dh_room == 0 ? 0 : head_dh_splits(tiles, slabs, L.dh_room), L.g_cached, L.dw_cached,
                    L.dw_tile.tp, L.dw_tile.tq, L.dw_splits, L.dh_tile.tp,
                    (long long)L.t_pad);
    }
    return 0;
}
