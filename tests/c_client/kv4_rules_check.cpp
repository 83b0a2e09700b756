// Prints what kv4_rules.h says of calls.  Input, a call a line: rows of a key head, bf16, SMs, requests, key heads,
// tiles that the block table holds, largest cluster.  Output: rows of a block, cluster, grid, CTAs with a full share.
#include <cstdio>

#include "kv4_rules.h"

using namespace attn;

int main() {
  int R, bf16, sms, B, H, most;
  long long tiles;
  while (std::scanf("%d %d %d %d %d %lld %d", &R, &bf16, &sms, &B, &H, &tiles, &most) == 7) {
    const int rp = kv4_rows(R, bf16), n_rb = (R + rp - 1) / rp;
    const long long segs = (long long)B * H * n_rb;
    const int c = kv4_cluster(rp, bf16, sms, B, segs, tiles, most);
    const int grid = c ? (int)(segs * c) : kv4_grid(rp, bf16, sms, segs * tiles);
    std::printf("%d %d %d %d\n", rp, c, grid, kv4_full(rp, bf16, sms, grid));
  }
}
