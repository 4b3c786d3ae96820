// Host-only check of how the prompt kernel finds the tiles in which it looks for NaN values
// (segment_span in attn_cache_prompt.cu) against counting them one by one, with the
// compiler's check of signed arithmetic.  Compiled and run by tests/test_prompt_nan.py;
// nothing is launched on a GPU.
#include "attn_cache_prompt.cu"

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
    std::printf("checked %d bad %d\n", checked, bad);
    return bad != 0;
}
