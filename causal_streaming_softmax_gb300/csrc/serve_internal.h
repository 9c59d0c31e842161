// serve_internal.h - what the host API of the packed and paged calls hands
// their kernel launchers: validated sizes and strides.
#pragma once

#include "attn_internal.h"

namespace css {

// A token-major tensor of 64-wide head rows: (token, head) at
// base + token * t + head * h (elements).
struct RowsArg {
  void* p;
  long long t, h;
};

// A pool of pages: (page, head, row) at base + page * pg + head * h + row * r.
struct PoolArg {
  void* p;
  long long pg, h, r;
};

struct PackedDims {
  int tokens, batch, H, Hkv, G, causal, bf16;
  float c;  // fp32(scale / ln 2)
};

struct PagedDims {
  int batch, tokens, H, Hkv, G, pages, width, shift /* log2 page size */, max_new, bf16;
  float c;
};

int launch_packed_fwd(const PackedDims& d, const DevCtx& ctx, const RowsArg& q, const RowsArg& k,
                      const RowsArg& v, const int32_t* cu, const RowsArg& o, float* lse,
                      cudaStream_t stream);
int launch_paged_plan(const PagedDims& d, const DevCtx& ctx, const int32_t* cached,
                      const int32_t* fresh, int32_t* ring, const int32_t* state, int32_t* table,
                      int32_t* cu, int32_t* lens, int32_t* slots, int32_t* next,
                      cudaStream_t stream);
int launch_paged_store(const PagedDims& d, const DevCtx& ctx, const RowsArg& k, const RowsArg& v,
                       const int32_t* slots, const PoolArg& kc, const PoolArg& vc,
                       cudaStream_t stream);
size_t paged_workspace_bytes(const PagedDims& d);
int launch_paged_fwd(const PagedDims& d, const DevCtx& ctx, const RowsArg& q, const PoolArg& kc,
                     const PoolArg& vc, const int32_t* table, const int32_t* cu,
                     const int32_t* lens, void* ws, const RowsArg& o, float* lse,
                     cudaStream_t stream);

}  // namespace css
