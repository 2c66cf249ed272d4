// Host check of the sinks part of mask.cuh and dq_order.cuh against a scan of
// the mask: which query rows see a key, which query blocks a key block visits,
// which key blocks a query block visits (its sinks, then its window), and that
// the deterministic backward's turns of every dQ tile are 0, 1, ..., K - 1.
#include <algorithm>
#include <cstdio>
#include <vector>

#include "kernels.h"
#include "mask.cuh"
#include "dq_order.cuh"

using namespace attn;

struct HostTile {
    int b, n, lq, lk, q_row0;
    const unsigned char* mcol;
};

static long bad = 0;

static void check(int lq, int lk, int wl, int wr, int sinks) {
    const MaskBand m = mask_band(lq, lk, wl, wr, sinks);
    auto sees = [&](int i, int j) {
        const int d = lk - lq;
        return !(wr >= 0 && j > i + d + wr) && (j >= i + d - wl || j < sinks);
    };
    auto block_sees = [&](int q, int n) {
        for (int i = q * 128; i < std::min(lq, q * 128 + 128); ++i)
            for (int j = n * 128; j < std::min(lk, n * 128 + 128); ++j)
                if (sees(i, j)) return true;
        return false;
    };
    const int nq = (lq + 127) / 128, nk = (lk + 127) / 128;
    for (int j = 0; j < lk; ++j)
        for (int i = 0; i < lq; ++i) bad += sees(i, j) != (i >= band_query_lo(m, j) && i < band_query_hi(m, j));
    for (int n = 0; n < nk; ++n) {
        int lo, hi;
        band_query_blocks(m, n * 128, n * 128 + 127, 128, &lo, &hi);
        for (int q = 0; q < nq; ++q) bad += block_sees(q, n) != (q >= lo && q < hi);
    }
    BwdParams p{};
    p.g.causal = wr >= 0;
    p.g.win_left = wl;
    p.g.win_right = wr;
    p.mask = BlockMask{nullptr, 1, sinks};
    for (int q = 0; q < nq; ++q) {
        int lo, hi;
        const bool has = band_key_blocks(m, q * 128, q * 128 + 127, 128, &lo, &hi);
        const int n_sink = has ? band_sink_blocks(m, 128, lo) : 0;
        std::vector<int> turns;
        for (int n = 0; n < nk; ++n) {
            const bool any = block_sees(q, n);
            bad += any != (has && (n < n_sink || (n >= lo && n < hi)));
            if (any) turns.push_back(dq_turn<true, false>(p, HostTile{0, n, lq, lk, 0, nullptr}, 0, q));
        }
        std::sort(turns.begin(), turns.end());
        for (int k = 0; k < (int)turns.size(); ++k) bad += turns[k] != k;
    }
}

int main() {
    for (int lq : {1, 100, 128, 129, 300, 513})
        for (int lk : {1, 77, 128, 300, 513, 700})
            for (int wl : {0, 5, 127, 128, 200})
                for (int wr : {-1, 0, 3, 64})
                    for (int sinks : {1, 4, 128, 129, 300, 1000}) check(lq, lk, wl, wr, sinks);
    printf("%ld disagreements\n", bad);
    return bad != 0;
}
