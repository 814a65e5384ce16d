// The addresses of the 256 x 256 tiles' loads (csrc/fp8_panel.h) against the rows that they may read, for
// tiles of every number of rows: a load that the buffer's range check lets through lies inside the operand,
// and is the row and block that was meant, whichever way the check treats the scalar offset.
#include <cstdint>
#include <cstdio>

#include "fp8_panel.h"

using muon::Panel;

// The ways in which a range check may treat vector offset v and scalar offset s of a buffer of n bytes.
static bool passes(int how, int64_t v, int64_t s, int64_t n) {
    switch (how) {
        case 0: return v + s < n;
        case 1: return v < n - s;                             // signed: never where s > n
        case 2: return v < (int64_t)(uint32_t)(n - s);        // unsigned: always where s > n
        default: return v < n;                                // the scalar offset takes no part
    }
}

static int64_t check(int32_t rows, int32_t ld, int32_t kp, bool row_in_scalar) {
    const int32_t size = Panel::bytes(rows, ld, kp), blocks = kp / 128;
    if (size <= 0) return -1;
    int64_t outside = 0;
    const int32_t steps[3] = {0, blocks / 2, blocks - 1};
    for (int how = 0; how < 4; ++how)
        for (int32_t kb : steps)
            for (int32_t r = 0; r < 256; ++r)
                for (int32_t c = 0; c < 8; ++c) {
                    // 64 rows an instruction
                    int64_t v = Panel::lane(r % 64, c, ld), s = Panel::block(kb);
                    (row_in_scalar ? s : v) += Panel::rows(r / 64 * 64, ld);   // in s: how it must not be
                    if (v < 0 || v + s > 0x7fffffff || s > 0x7fffffff) return -1;
                    const bool in = passes(how, v, s, size);
                    if (in && v + s + 16 > size) ++outside;
                    if (!row_in_scalar && in != (r < rows)) return -1;
                    if (in && r < rows && v + s != (int64_t)r * ld + 128 * (int64_t)kb + 16 * c) return -1;
                }
    return outside;
}

int main() {
    const int32_t kps[] = {128, 256, 4096, 8388352};
    for (int32_t rows = 1; rows <= 256; ++rows)
        for (int32_t kp : kps)
            for (int32_t more = 0; more <= 4096; more = 16 * (17 * more / 16 + 1)) {
                const int32_t ld = kp + more;
                if (ld >= 1 << 23) continue;
                if (check(rows, ld, kp, false) != 0) {
                    std::printf("rows %d ld %d kp %d: a load outside, or not the row that was meant\n", rows, ld, kp);
                    return 1;
                }
                // the check itself tells the two apart
                if (rows <= 192 && check(rows, ld, kp, true) <= 0 && ld < 1 << 20) {
                    std::printf("rows %d ld %d kp %d: the planted mistake is not seen\n", rows, ld, kp);
                    return 1;
                }
            }
    std::puts("panels ok");
    return 0;
}
