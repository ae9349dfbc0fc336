"""The scale of an E2M1 row in csrc/unit_codes.h: a product with fl32(1 / 6) and one correction is
fl32(amax / 6) for every significand (no GPU: binary32 and its fused multiply-add are the same here).
Powers of two change nothing while all values are normal."""
import subprocess

SOURCE = r"""
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>
int main(void) {
    const float top = 6.0f, r = 1.0f / 6.0f;
    long wrong = 0;
    for (uint32_t e = 27; e <= 247; e += 110)  /* 2^-100, 2^10, 2^120 */
        for (uint32_t m = 0; m < 1u << 23; m++) {
            if (e == 247 && m) break;  /* up to 2^120 */
            const uint32_t u = e << 23 | m;
            float amax;
            memcpy(&amax, &u, 4);
            const float q = amax * r;
            wrong += fmaf(fmaf(-q, top, amax), r, q) != amax / top;
        }
    printf("%ld", wrong);
    return 0;
}
"""


def test_every_significand(tmp_path):
    (tmp_path / "d.c").write_text(SOURCE)
    subprocess.check_call(["gcc", "-O2", "-mfma", "-ffp-contract=off", str(tmp_path / "d.c"), "-o", str(tmp_path / "d"), "-lm"])
    assert subprocess.check_output([str(tmp_path / "d")]) == b"0"
