// Host check of where the linear attention walk finds its operands' rows
// (nonlinear_rnn_solve_pararnn_amd/csrc/walk_rows.hpp), built by
// tests/test_walk_rows.py.  Prints "ok" and exits 0 when every check passes.
//
// Every thread's loads of every chunk are gone through with the header's own
// offsets, for both directions, element sizes and alignments, rows that are
// dense, spaced, shared and overlapping: what the groups put into the tile has
// to be the chunk's elements and zeros elsewhere, and no word is touched that
// holds none of the tensor's bytes.
#include <stdint.h>
#include <stdio.h>

#include <algorithm>
#include <vector>

#include "walk_rows.hpp"

using namespace prn::walk;

static long fails = 0, seen = 0;
static void fail(const char *what, int W, int C, int es, int d, int c0, long st, int rev, int cnt, int skew, int r, int c) {
    if (fails++ < 20)
        fprintf(stderr, "FAIL %s: W=%d C=%d bytes=%d d=%d c0=%d stride=%ld rev=%d cnt=%d skew=%d row %d column %d\n", what, W, C, es, d,
                c0, st, rev, cnt, skew, r, c);
}

// A tensor of L rows of d elements of es bytes, `st` elements apart, `skew`
// bytes into a word; an element's two-byte pieces hold their own places, and
// what lies around the tensor is marked.
struct Memory {
    uintptr_t lo, hi;
    uint32_t half(uintptr_t at) const { return at >= lo && at < hi ? (uint32_t)(1 + (at - lo) / 2 % 65000) : 65535u; }
    uint32_t word(uintptr_t at) const { return half(at) | half(at + 2) << 16; }
};

template <int W, int C>
static void check(int es, bool vec, int d, int c0, long st, int rev, int64_t L, int skew) {
    const uintptr_t base = 0x100000 + skew;
    const Memory mem{base, base + (uintptr_t)(((L - 1) * st + d) * es)};
    const uint32_t tail = (uint32_t)((d - c0) * es);
    const Rows v = rows_from(reinterpret_cast<const char *>(base + (uintptr_t)c0 * es), st * es, tail, L, 0, C, rev);
    const int chunks = (int)((L + C - 1) / C), last = (int)(L - (int64_t)(chunks - 1) * C);
    std::vector<uint32_t> tile((size_t)C * W * es / 2);
    for (int i = 0; i <= chunks; ++i) {  // one past the last: nothing to read
        const int cnt = i < chunks - 1 ? C : i == chunks - 1 ? last : 0;
        const char *first = v.at(i, cnt, C);
        const uint32_t sk = !vec && es == 2 ? Rows::word_skew(first) : 0u;
        const uint32_t size = !vec && es == 2 ? v.word_bytes(sk, cnt) : v.bytes(cnt);
        const uintptr_t buf = (uintptr_t)first - sk;
        auto read = [&](uint32_t o) {
            if ((uint64_t)o + 4 > size) return 0u;
            const uintptr_t at = buf + o;
            if (at + 4 <= mem.lo || at >= mem.hi) fail("a word of others", W, C, es, d, c0, st, rev, cnt, skew, -1, -1);
            return mem.word(at);
        };
        std::fill(tile.begin(), tile.end(), 0xffffffffu);
        for (int t = 0; t < kThreads; ++t) {
            Groups<W, C> g;
            g.init(v, es, t);
            for (int n = 0; n < g.kN; ++n) {
                const int r = g.row(n), c = g.column(n), words = 2 * es;
                if (r >= C) continue;
                uint32_t x[9] = {}, u[8];
                if (vec) {
                    const uint32_t o = g.offset(v, n, v.shift(cnt, C));
                    const int per = 16 / es;
                    for (int h = 0; h < 8 / per; ++h)
                        for (int k = 0; k < 4; ++k)
                            u[4 * h + k] = read((h == 0 ? o : (c + h * per < g.left ? o + 16 * h : kNowhere)) + 4 * k);
                } else {
                    const uint32_t shift = v.shift(cnt, C) - sk, o = g.offset(v, n, shift) & ~3u;
                    for (int k = 0; k < words + (es == 2); ++k) x[k] = read(o + 4 * k);
                    const uint32_t bits = es == 2 ? (g.offset(v, n, shift) & 2u) << 3 : 0u;
                    for (int k = 0; k < words; ++k)
                        u[k] = g.own_word((uint32_t)(((uint64_t)x[k + 1] << 32 | x[k]) >> bits), k, es, g.own(n));
                }
                for (int k = 0; k < words; ++k) u[k] = !vec && g.past(t, n, cnt) ? 0u : u[k];
                for (int k = 0; k < words; ++k)
                    for (int h = 0; h < 2; ++h) tile[((size_t)r * W + c) * es / 2 + 2 * k + h] = u[k] >> (16 * h) & 0xffffu;
            }
        }
        for (int r = 0; r < C; ++r)
            for (int c = 0; c < W; ++c)
                for (int h = 0; h < es / 2; ++h) {
                    const bool mine = r < cnt && c < d - c0;
                    const int64_t t = rev ? L - 1 - ((int64_t)i * C + r) : (int64_t)i * C + r;
                    const uint32_t want = mine ? mem.half(base + (uintptr_t)((t * st + c0 + c) * es + 2 * h)) : 0u;
                    ++seen;
                    // rows that all lie at one place are their own copies past the end, and as little finite as the others
                    if (st == 0 && vec && r >= cnt) continue;
                    if (tile[((size_t)r * W + c) * es / 2 + h] != want) fail("an element", W, C, es, d, c0, st, rev, cnt, skew, r, c);
                }
    }
}

template <int W, int C>
static void widths(int es) {
    const int lo = W == 32 ? 1 : W == 64 ? 33 : W == 96 ? 65 : W == 128 ? 97 : 129;
    for (int d : {lo, lo + 1, lo + 7, lo + 12, (lo + W) / 2, W - 7, W - 1, W})
        for (int64_t L : {(int64_t)1, (int64_t)13, (int64_t)C, (int64_t)(C + 13), (int64_t)(2 * C - 1)})
            for (long st : {(long)d, (long)d + 1, (long)d + 8, (long)d * 3, (long)d - 1, (long)d / 2, 1L, 0L})
                for (int rev = 0; rev < 2; ++rev) {
                    if (st < 0) continue;
                    for (int skew = 0; skew < 4; skew += es) check<W, C>(es, false, d, 0, st, rev, L, skew);
                    const int n = 16 / es;
                    if (d % n == 0 && st % n == 0 && (st >= d || st == 0)) check<W, C>(es, true, d, 0, st, rev, L, 0);
                }
}

int main() {
    for (int es : {2, 4}) {
        widths<32, 32>(es);
        widths<64, 32>(es);
        widths<96, 32>(es);
        widths<128, 32>(es);
        widths<256, 32>(es);
        if (es == 2) {
            widths<32, 64>(es);
            widths<64, 64>(es);
            widths<96, 64>(es);
            widths<128, 64>(es);
            widths<256, 64>(es);
        }
        // later column blocks of a wide operand
        for (int d : {77, 101, 130, 193, 255})
            for (int c0 = 0; c0 < d; c0 += 64)
                for (long st : {(long)d, (long)d + 3})
                    for (int rev = 0; rev < 2; ++rev)
                        for (int skew = 0; skew < 4; skew += es) {
                            if (d - c0 > 64) continue;
                            check<64, 32>(es, false, d, c0, st, rev, 45, skew);
                            check<64, 64>(es, false, d, c0, st, rev, 77, skew);
                        }
    }
    if (fails == 0) printf("ok\n");
    else fprintf(stderr, "%ld of %ld\n", fails, seen);
    return fails != 0;
}
