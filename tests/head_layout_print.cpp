// How calls of the output-head losses are cut, for the tests: reads lines of
// "tokens hidden vocab top_k dtype backward" and prints the layout of each as
// name=value pairs (head_layout.cpp, linked in).
#include <cstdio>

#include "head_layout.h"

using namespace dmuon;

int main() {
    long long t, d, v;
    int k, dt, back;
    while (std::scanf("%lld %lld %lld %d %d %d", &t, &d, &v, &k, &dt, &back) == 6) {
        const dmuon_head_desc desc{t, d, v, k, dt};
        if (head_check_desc(&desc) != DMUON_OK) {
            std::printf("refused=1\n");
            continue;
        }
        const HeadLayout L = head_layout_of(desc, back != 0);
        std::printf("refused=0 s_tp=%d s_tq=%d dh_tp=%d dh_tq=%d dw_tp=%d dw_tq=%d splits=%d dw_splits=%d pieces=%d "
                    "piece=%lld pack=%d stream=%d low=%d keep=%d t_pad=%lld bytes=%zu s_slots=%d dh_slots=%d dw_slots=%d\n",
                    L.s_tile.tp, L.s_tile.tq, L.dh_tile.tp, L.dh_tile.tq, L.dw_tile.tp, L.dw_tile.tq, L.splits,
                    L.dw_splits, L.pieces, (long long)L.piece, L.pack_weight, L.stream_weight, L.low, L.keep_logits,
                    (long long)L.t_pad, L.bytes, head_slots(L.s_tile.tp), head_slots(L.dh_tile.tp),
                    head_slots(L.dw_tile.tp));
    }
    return 0;
}
