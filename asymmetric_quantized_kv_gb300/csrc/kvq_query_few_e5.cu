// The few-row attention kernels over E5M2 caches (a translation unit a format, compiled in parallel).
#include "kvq_query_few.cuh"

namespace kvq {

kvq_status launch_query_few_e5(const KvqView& v, const QueryArgs& a, void* ws, cudaStream_t st) {
  return launch_few_format<kE5>(v, a, ws, st);
}

}  // namespace kvq
