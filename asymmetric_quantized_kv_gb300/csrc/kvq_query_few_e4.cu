// The few-row attention kernels over E4M3 caches (a translation unit a format, compiled in parallel).
#include "kvq_query_few.cuh"

namespace kvq {

kvq_status launch_query_few_e4(const KvqView& v, const QueryArgs& a, void* ws, cudaStream_t st) {
  return launch_few_format<kE4>(v, a, ws, st);
}

}  // namespace kvq
