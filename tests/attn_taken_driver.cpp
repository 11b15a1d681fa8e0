// Where new tokens go, by the rule that the writing kernel shares with the host.
// Input on stdin: "<start> <n> <len> <w>" a line; output "<block> <lo> <hi>".
#include <cinttypes>
#include <cstdio>

#include "../sparse_dense_matrix_amd/csrc/attn.h"

int main() {
  int64_t start;
  int32_t n, len;
  uint32_t w;
  while (std::scanf("%" SCNd64 " %" SCNd32 " %" SCNd32 " %" SCNu32, &start, &n, &len, &w) == 4) {
    const sdm::AttnTaken x = sdm::attn_taken(start, n, len, w);
    std::printf("%d %d %d\n", x.id, x.lo, x.hi);
  }
  return 0;
}
