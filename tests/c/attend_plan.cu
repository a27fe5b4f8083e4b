// Host-side check of the attention calls' plan, without a GPU: includes the
// query calls' source, makes handles by hand and prints what a call would
// launch.  One plan a line of standard input:
//   sm_count clusters[4] kv_heads head_dim | tokens requests max_q_len blocks shared_len heads | block_size
// and one line of results: wide shared units splits key_parts parts shared_units ml_bytes o_bytes
#include "query.cu"

#include <cstdio>

int main(int argc, char**) {
  if (argc > 1) {  // the cluster counts that a GPU's answers make
    for (int largest : {8, 4, 2, 1, 0}) {
      int64_t clusters[4] = {7, 7, 7, 7};
      const bool ok = count_clusters(clusters, [&](unsigned ctas, int* n) {
        *n = int(ctas) <= largest ? 16 / int(ctas) : 0;
        return int(ctas) > 2 * largest ? cudaErrorInvalidValue : cudaSuccess;
      });
      std::printf("%d %d %d %d %d\n", int(ok), int(clusters[0]), int(clusters[1]), int(clusters[2]), int(clusters[3]));
    }
    return 0;
  }
  is_query q;
  long long c[4];
  is_attend_t a{};
  is_cache_t cache{};
  while (std::scanf("%d %lld %lld %lld %lld %d %d %d %d %d %d %d %d %d", &q.sm_count, &c[0], &c[1], &c[2], &c[3],
                    &q.kv_heads, &q.head_dim, &a.num_tokens, &a.num_requests, &a.max_q_len, &a.max_blocks_per_req,
                    &a.shared_len, &a.q.num_heads, &cache.block_size) == 14) {
    for (int i = 0; i < 4; ++i) q.clusters[i] = c[i];
    const AttendPlan p = plan_attend(&q, &a, &cache);
    std::printf("%d %d %lld %d %d %d %lld %lld %lld\n", int(p.wide), int(p.shared), (long long)p.units, p.splits,
                p.key_parts, p.parts, (long long)p.shared_units, (long long)p.ml_bytes, (long long)p.o_bytes);
  }
  return 0;
}
