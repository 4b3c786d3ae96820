// Host-only check of how the prompt kernel finds the tiles in which it looks for NaN values,
// with the compiler's check of signed arithmetic: segment_span in attn_cache_prompt.cu against
// counting tiles one by one; PromptUnit::all_see against the mask's definition for every row
// and token, and the number of tiles that not every row sees, which bounds the look.  Compiled and run by tests/test_prompt_nan.py;
// nothing is launched on a GPU.
#include "attn_cache_prompt.cu"

#include <algorithm>
#include <cstdio>
#include <initializer_list>

using namespace attn;

int main() {
    int checked = 0, bad = 0;
    for (int t0 : {0, 1, 7, 1 << 23})
        for (int v0 : {0, 1, 5, 8000000})
            for (int n : {1, 2, 9})
                for (int lo : {INT_MAX, 0, 1, 6, 7, 8, 12, (1 << 23) - 1, 1 << 23, (1 << 23) + 3})
                    for (int len : {-1, 0, 1, 3, 100}) {
                        const int hi = lo == INT_MAX ? -1 : lo + len;
                        const TileSpan s = segment_span(lo, hi, t0, v0, v0 + n);
                        bool ok = v0 <= s.first && s.end <= v0 + n;
                        for (int i = 0; i < n; ++i) {
                            const bool in = lo <= t0 + i && t0 + i <= hi;
                            ok = ok && in == (s.first <= v0 + i && v0 + i < s.end);
                        }
                        ++checked;
                        bad += !ok;
                        if (!ok) std::printf("t0 %d v0 %d n %d lo %d hi %d: %d %d\n", t0, v0, n, lo, hi, s.first, s.end);
                    }
    int most = 0;
    long long some = 0, whole = 0, missed = 0;
    for (int q_len : {1, 9, 65, 300, 700})
        for (int G : {1, 3, 8, 16})
            for (int len : {1, 64, 129, 300, 700, 2500})
                for (int left : {-1, 0, 20, 127, 128, 140, 600})
                    for (int sinks : {0, 1, 128, 200}) {
                        CacheFwdParams p = {};
                        p.c.seq_lens = &len;
                        p.c.page_size = 16;
                        p.c.max_pages = 200;
                        p.H = G;
                        p.Hk = 1;
                        p.T = q_len;
                        p.left = left;
                        p.sinks = left < 0 ? 0 : sinks;
                        for (int pair = 0; pair * kPairRows < q_len * G; ++pair) {
                            const PromptUnit u = prompt_unit(p, 0, pair);
                            int edge = 0;
                            for (int t = 0; t < u.n; ++t) {
                                bool all = true;
                                for (int r = pair * kPairRows; r < std::min(u.rows, (pair + 1) * kPairRows) && all; r += 1) {
                                    const int pos = u.first_pos + r / G;
                                    for (int j = u.tile(t) * kTile; j < (u.tile(t) + 1) * kTile; ++j)
                                        all = all && j <= pos && (left < 0 || j >= pos - left || j < p.sinks);
                                }
                                ++checked;
                                // (a tile of which the window's edge meets the last sink may count as not seen by all)
                                const bool said = u.all_see(t, p.left, p.sinks);
                                bad += said && !all;
                                missed += all && !said;
                                edge += !said;
                                (said ? whole : some) += 1;
                            }
                            most = std::max(most, edge);
                        }
                    }
    std::printf("tiles that all rows see %lld, that not all see %lld, at most %d a walk\n", whole, some, most);
    bad += most > 7 || whole == 0 || some == 0 || missed * 100 > whole;
    std::printf("checked %d bad %d\n", checked, bad);
    return bad != 0;
}
