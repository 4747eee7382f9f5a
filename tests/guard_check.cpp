// Host-side check of the prompt attention guard's split of a value tile between
// its two warps (mk_ops.h): every vector of the tile is looked at exactly once,
// a warp's vectors hold its own half of the columns and nothing of the other's
// (so the two share no word they write), the swizzle is undone, and eight lanes
// in a row read different banks.  Prints "ok" or the first violation.
#include <cstdio>
#include "../persistent_decode_megakernel_02_b200/csrc/mk_ops.h"

using namespace mk;

int main() {
    for (int d = 64; d <= 128; d += 64) {
        static int seen[2048];
        for (int i = 0; i < 2048; ++i) seen[i] = 0;
        const int steps = 128 * d * 2 / 16 / 64;
        for (int half = 0; half < 2; ++half)
            for (int step = 0; step < steps; ++step) {
                for (int lane = 0; lane < 32; ++lane) {
                    const int v = guard_vector(d, half, step, lane);
                    if (v < 0 || v >= 128 * d / 8) { printf("d %d: vector %d out of the tile\n", d, v); return 1; }
                    if (seen[v]++) { printf("d %d: vector %d twice\n", d, v); return 1; }
                    const int row = guard_row(v), col = guard_column(v);
                    // where the tile copy puts (row, col): rows of 128 bytes, 16-byte
                    // chunks exchanged by the row's low three bits
                    const int at = col / 64 * 1024 + row * 8 + ((col % 64 / 8) ^ (row & 7));
                    if (at != v) { printf("d %d: vector %d is not (%d, %d)\n", d, v, row, col); return 1; }
                    if (col / (d / 2) != half) { printf("d %d: column %d by warp %d\n", d, col, half); return 1; }
                }
                for (int group = 0; group < 4; ++group) {
                    int banks = 0;
                    for (int i = 0; i < 8; ++i) banks |= 1 << guard_vector(d, half, step, group * 8 + i) % 8;
                    if (banks != 255) { printf("d %d: banks %x\n", d, banks); return 1; }
                }
            }
        for (int i = 0; i < 128 * d / 8; ++i)
            if (!seen[i]) { printf("d %d: vector %d never\n", d, i); return 1; }
    }
    printf("ok\n");
    return 0;
}
