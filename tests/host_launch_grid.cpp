// Host check of the grids that launches get (grid_of, xcd_grid_of and launch_grid in
// zr_internal.hpp): any number of workgroups of any size stays below 2^32 work items in
// the dimension, a grid that fits is left as it is, and grids dealt to the XCDs stay
// multiples of 8.  Prints "ok: <count>".
#include <cstdint>
#include <cstdio>

#include "zr_internal.hpp"

static int fails = 0;

static void check(bool c, const char *what, int64_t blocks, unsigned threads, unsigned x)
{
    if (!c && fails++ < 20)
        std::printf("FAIL %s: %lld workgroups of %u -> %u\n", what, (long long)blocks, threads, x);
}

int main()
{
    const unsigned threads[] = {1, 64, 128, 192, 256, 512, 1024};
    long count = 0;
    for (unsigned t : threads) {
        const dim3 block(t);
        for (int shift = 0; shift < 60; ++shift)
            for (int64_t off = -17; off <= 17; ++off) {
                const int64_t blocks = (int64_t(1) << shift) + off;
                if (blocks < 1)
                    continue;
                for (const bool xcd : {false, true}) {
                    const dim3 asked = xcd ? zr::xcd_grid_of(blocks) : zr::grid_of(blocks);
                    const dim3 got = zr::launch_grid(asked, block);
                    check((uint64_t)got.x * t < (uint64_t(1) << 32), "work items", blocks, t, got.x);
                    check(got.x >= 1 && got.x <= asked.x && got.y == 1 && got.z == 1, "range", blocks, t, got.x);
                    check((uint64_t)(asked.x + 8u) * t >= (uint64_t(1) << 32) || got.x == asked.x, "kept", blocks, t, got.x);
                    check((uint64_t)(got.x + 8u) * t >= (uint64_t(1) << 32) || got.x == asked.x, "as many as fit", blocks, t, got.x);
                    check(!xcd || got.x % 8 == 0, "multiple of 8", blocks, t, got.x);
                    ++count;
                }
            }
    }
    if (fails) {
        std::printf("%d failures\n", fails);
        return 1;
    }
    std::printf("ok: %ld grids\n", count);
    return 0;
}
