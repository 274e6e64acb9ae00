// The few-row attention kernels over INT8 caches (a translation unit a format, compiled in parallel).
#include "kvq_query_few.cuh"

namespace kvq {

kvq_status launch_query_few_i8(const KvqView& v, const QueryArgs& a, void* ws, cudaStream_t st) {
  return launch_few_format<kI8>(v, a, ws, st);
}

}  // namespace kvq
