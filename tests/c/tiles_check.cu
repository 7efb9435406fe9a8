/* The 32-bit arithmetic that cuts groups of rows into token tiles, against 64 bits,
 * on the host: every row of a group of any size up to 2^31 - 1 has its tile. */
#include <cstdio>
#include <initializer_list>

#include "mxfp4_tiles.cuh"

namespace mx = moe::mx;
typedef long long ll;

static int failures = 0;

static void group(ll rows, int cap) {
  const ll tiles = mx::token_tiles(static_cast<int>(rows), cap);
  bool ok = tiles == (rows + cap - 1) / cap;
  if (ok && rows > 0) {
    const ll size = mx::tile_size(static_cast<int>(rows), static_cast<int>(tiles));
    ok = size > 0 && size <= cap && size % 16 == 0 && (tiles - 1) * size < rows && tiles * size >= rows;
  }
  if (!ok && ++failures <= 10) printf("FAILED: %lld rows in tiles of at most %d\n", rows, cap);
}

static void half(ll row, int n, ll R) {
  const ll second = row + n / 2 < R ? row + n / 2 : R;
  const bool ok = mx::half_row(static_cast<int>(row), n, 0, static_cast<int>(R)) == row &&
                  mx::half_row(static_cast<int>(row), n, 1, static_cast<int>(R)) == second;
  if (!ok && ++failures <= 10) printf("FAILED: half of %d columns at row %lld of %lld\n", n, row, R);
}

int main() {
  const ll most = (1ll << 31) - 1;
  for (int cap = 16; cap <= 256; cap += 16) {
    for (ll rows = 0; rows <= 1100; ++rows) group(rows, cap);
    for (ll near : {1ll << 16, 1ll << 24, 1ll << 30, most * cap / (cap + 1), most - cap, most - 300})
      for (ll rows = near - 300; rows <= near + 300; ++rows)
        if (rows <= most) group(rows, cap);
  }
  for (ll R : {1ll, 17ll, 300ll, 1ll << 30, most - 8, most})
    for (ll row = R > 300 ? R - 300 : 0; row < R; ++row)
      for (int n = 16; n <= 256; n += 16) half(row, n, R);
  if (failures == 0) printf("tiles ok\n");
  return failures != 0;
}
