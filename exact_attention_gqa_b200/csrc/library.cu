// The library's translation unit: the attention entry points, then the 8-bit paged cache
// with block scales, which uses their argument checks and device table.  (One unit,
// because the kernels share the device error word.)
#include "gqa_attn.cu"
#include "kv8_host.cuh"
