// Host check of the offsets that the large product's prefetch loads from (group_of_row in
// fp8.hpp): a lane that is switched off stays off in every group, and the others'
// offsets are their row's.  Prints "ok: <count>".
#include <cstdio>

#include "fp8.hpp"

int main()
{
    long count = 0, fails = 0;
    const uint32_t rows[] = {0, 16, 4096, 255u * 8388592u};
    for (int32_t kb : {2, 3, 32, 65536})
        for (int32_t g = 0; g <= kb + 1; ++g) {
            fails += zr::group_of_row(zr::kNowhere, g, kb) != zr::kNowhere;
            for (uint32_t row : rows)
                fails += zr::group_of_row(row, g, kb) != (g < kb ? row + 128u * (uint32_t)g : zr::kNowhere);
            ++count;
        }
    if (fails) {
        std::printf("%ld failures\n", fails);
        return 1;
    }
    std::printf("ok: %ld cases\n", count);
    return 0;
}
