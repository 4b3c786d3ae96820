// Host-only check of the backward with sinks (sink_parts_for and BwdWork::split_at in
// attn_bwd.cu): on 152 SMs, for both head dimensions, every step (query head, query tile) of
// every key tile is in exactly one item or part, no part is empty, parts fit the workspace, and
// the shapes that are meant to be split are.  Compiled and run by tests/test_sink_parts.py;
// nothing is launched on a GPU.
#include "attn_bwd.cu"

#include <cstdio>
#include <set>
#include <utility>

using namespace attn;

namespace {
int checked = 0, bad = 0;

// Parts of a sink tile.
int check(int D, int B, int H, int Hk, int N, int left, int right, int sinks) {
    BwdParams p{};
    p.N = N;
    p.H = H;
    p.Hk = Hk;
    p.BHk = B * Hk;
    p.n_kv = (N + kTile - 1) / kTile;
    p.win_left = left;
    p.win_right = right;
    p.sinks = sinks < N ? sinks : N;
    p.sink_tiles = (p.sinks + kTile - 1) / kTile;
    const long long sink_items = static_cast<long long>(p.BHk) * p.sink_tiles, room = sink_items * kBwdSinkParts;
    p.split_cap = static_cast<int>(room < kBwdSinkCap ? room : kBwdSinkCap);
    const int items = p.BHk * p.n_kv, G = H / Hk;
    p.split_base = items;
    p.split_parts = 1;
    sink_parts_for(D, 152, &p);
    int wrong = 0;
    const int all = p.split_base + (items - p.split_base) * p.split_parts;
    std::set<int> slots;
    std::set<std::pair<long long, int>> steps;  // (key tile of a head, step)
    for (int v = 0; v < all; ++v) {
        const auto w = BwdWork<true>::split_at(p, v);
        if (v >= p.split_base) {
            wrong += w.n_steps < 1 || w.slot < 0 || w.slot >= p.split_cap || w.j * kTile >= p.sinks;
            wrong += !slots.insert(w.slot).second;
        } else {
            wrong += w.slot != -1;
        }
        int bh = w.bh_first, tt = w.tt0;
        for (int t = 0; t < w.n_steps; ++t, ++tt) {
            if (tt == w.n_qh) tt = 0, ++bh;
            wrong += bh < w.q_bh0 || bh >= w.q_bh0 + G || w.q_tile(tt) >= p.n_kv;
            wrong += !steps.insert({static_cast<long long>(w.kv_bh) * p.n_kv + w.j, bh * p.n_kv + w.q_tile(tt)}).second;
        }
    }
    long long want = 0;  // steps that hold a visible pair of tiles
    for (int j = 0; j < p.n_kv; ++j)
        for (int i = 0; i < p.n_kv; ++i) {
            const int q1 = std::min(N, (i + 1) * kTile) - 1, k0 = j * kTile, k1 = std::min(N, k0 + kTile) - 1;
            const bool ahead = right < 0 || k0 <= q1 + right, behind = k1 >= i * kTile - left || k0 < p.sinks;
            want += ahead && behind ? static_cast<long long>(p.BHk) * G : 0;
        }
    wrong += static_cast<long long>(steps.size()) != want;
    ++checked;
    bad += wrong != 0;
    if (wrong) std::printf("D %d B %d H %d Hk %d N %d left %d right %d sinks %d: %d parts, wrong %d\n", D, B, H, Hk, N, left,
                           right, sinks, p.split_parts, wrong);
    return p.split_parts;
}
}  // namespace

int main() {
    for (int D : {64, 128}) {
        for (int B : {1, 3})
            for (int H : {1, 2, 8, 40})
                for (int Hk : {1, 2, 8, 40}) {
                    if (Hk > H || H % Hk != 0) continue;
                    for (int N : {1, 129, 700, 2500, 8192})
                        for (int left : {0, 100, 255})
                            for (int right : {0, 140, -1})
                                for (int sinks : {1, 130, 513})
                                    if (left < N - 1) check(D, B, H, Hk, N, left, right, sinks);
                }
        // the shapes that tests/test_gpu_sinks.py takes for split and for whole
        struct { int B, H, Hk, N, left, sinks; } split[] = {{1, 2, 2, 8192, 200, 4}, {1, 8, 1, 2500, 255, 1},
                                                              {1, 40, 40, 4096, 100, 2}, {1, 2, 2, 6000, 130, 513}};
        for (const auto& c : split) {
            const int parts = check(D, c.B, c.H, c.Hk, c.N, c.left, 0, c.sinks);
            std::printf("D %d H %d Hk %d N %d sinks %d: %d parts\n", D, c.H, c.Hk, c.N, c.sinks, parts);
            bad += parts < 2;
        }
        bad += check(D, 5, 52, 52, 300, 100, 0, 4) != 1;
    }
    std::printf("checked %d bad %d\n", checked, bad);
    return bad != 0;
}
