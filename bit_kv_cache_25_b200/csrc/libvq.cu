// The translation unit of libvq: the block cache's entry points and kernels,
// then the paged cache's.
#include "vq_api.cu"

#include "paged_api.cuh"
