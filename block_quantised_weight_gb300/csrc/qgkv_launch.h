// Launchers of the qgkv.h operators; arguments are checked by kv_api.cu.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/qgkv.h"

namespace qg {

// Device address of the current device's status word; null if it cannot be had.
unsigned* status_ptr();

int launch_beam_select(const void* logits, int type, const float* cum, int requests, int beams, int64_t vocab,
                       int64_t row_stride, int keep, float* scores, int32_t* tokens, int32_t* parents,
                       uint8_t* workspace, cudaStream_t s);

int launch_append(const qgkv_cache& c, int64_t layer, const void* k, const void* v, int type, int64_t rows,
                  int64_t row_stride, int64_t head_stride, const int32_t* table, int64_t width, const int32_t* lens,
                  const int32_t* starts, int batch, unsigned* status, cudaStream_t s);

int launch_copy_pages(const qgkv_cache& c, const int32_t* src, const int32_t* dst, const int32_t* count, int64_t most,
                      unsigned* status, cudaStream_t s);
int launch_fork(const qgkv_cache& c, const int32_t* table, int64_t width, const int32_t* lens, int batch,
                const int32_t* parent, int batch2, const int32_t* refs, int32_t* table2, int32_t* lens2,
                int32_t* refs2, uint8_t* workspace, unsigned* status, cudaStream_t s);
int launch_compact(const qgkv_cache& c, const int32_t* table, int64_t width, const int32_t* lens, int batch,
                   const uint8_t* drop, const int32_t* refs, int32_t* table2, int32_t* lens2, int32_t* refs2,
                   int32_t* count, uint8_t* workspace, unsigned* status, cudaStream_t s);
int launch_reserve(int64_t pages, int page_tokens, int32_t* table, int64_t width, const int32_t* lens,
                   const int32_t* add, int batch, int32_t* refs, uint8_t* workspace, unsigned* status,
                   cudaStream_t s);
int launch_free(int64_t pages, int page_tokens, int32_t* table, int64_t width, int32_t* lens, const uint8_t* drop,
                int batch, int32_t* refs, unsigned* status, cudaStream_t s);

}  // namespace qg
