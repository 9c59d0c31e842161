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

// The parts of rows whose keys were split over blocks (serve_parts.cuh).
struct PartDesc {  // of a block's tail part: what it is and the block that ends it
  int q0, kv, rows, last;
};
struct PartArgs {
  float* o;    // [block][head, tail][rows][64]
  float2* ml;  // [block][head, tail][rows]
  PartDesc* desc;
  int rows;       // rows a part has room for
  int min_tiles;  // a block takes at least so many tiles
};

// Rows (new tokens x heads of a group) of a request that paged_decode takes,
// and the new tokens that makes for a group of G heads (0: none).
constexpr int kDecodeRows = 16;
constexpr int kMaxPagedBatch = 4096;
// Rows of a work item of the tile kernel: three tiles.
constexpr int kItemRows = 384;
int decode_tokens(int G);
// Whether paged_decode finishes every item itself (no parts to join).
bool decode_whole(const PagedDims& d, int sm_count);
int launch_paged_decode(const PagedDims& d, const DevCtx& ctx, const RowsArg& q,
                        const PoolArg& kc, const PoolArg& vc, const int32_t* table,
                        const int32_t* cu, const int32_t* lens, const PartArgs& part, int blocks,
                        const RowsArg& o, float* lse, cudaStream_t stream);
int launch_paged_rows(const PagedDims& d, const DevCtx& ctx, const RowsArg& q, const PoolArg& kc,
                      const PoolArg& vc, const int32_t* table, const int32_t* cu,
                      const int32_t* lens, const PartArgs& part, int blocks, int skip,
                      bool four, const RowsArg& o, float* lse, cudaStream_t stream);
// The same over a 4-bit cache (the pools' strides in bytes).
bool decode4_whole(const PagedDims& d, int sm_count);
int decode4_blocks(const PagedDims& d);  // a SM
int decode4_rows(const PagedDims& d);    // of an item, at most
int launch_paged_decode4(const PagedDims& d, const DevCtx& ctx, const RowsArg& q,
                         const PoolArg& kc, const PoolArg& vc, const int32_t* table,
                         const int32_t* cu, const int32_t* lens, const PartArgs& part, int blocks,
                         const RowsArg& o, float* lse, cudaStream_t stream);

// Lets `kernel` (known by an index of its own) use `bytes` of dynamic shared
// memory on the current device; set once a device.
enum {
  kSmemDecodeF16,
  kSmemDecodeBf16,
  kSmemWholeF16,
  kSmemWholeBf16,
  kSmemPackedF16,
  kSmemPackedBf16,
  kSmemRowsF16,
  kSmemRowsBf16,
  kSmemDecode4F16,
  kSmemDecode4Bf16,
  kSmemDecode4WholeF16,
  kSmemDecode4WholeBf16,
  kSmemDecode4WideF16,
  kSmemDecode4WideBf16,
  kSmemDecode4WideWholeF16,
  kSmemDecode4WideWholeBf16,
  kSmemDecode4SplitF16,
  kSmemDecode4SplitBf16,
  kSmemRows4F16,
  kSmemRows4Bf16,
  kSmemKernels
};
int allow_smem(int which, const void* kernel, size_t bytes);

// A rank-4 tiled tensor map of 64-wide 16-bit rows with the 128-byte swizzle:
// dimensions 64, d1, d2, d3, strides in elements, boxes 64 x b1 x b2 x b3.
bool encode_tmap_4d(CUtensorMap* map, bool bf16, const void* base, uint64_t d1, uint64_t d2,
                    uint64_t d3, uint64_t s1, uint64_t s2, uint64_t s3, uint32_t b1, uint32_t b2,
                    uint32_t b3);

// A rank-4 tiled tensor map of a 4-bit pool: a unit of eight rows, units of a page,
// heads, pages, boxes of `box` units.
bool encode_tmap_units(CUtensorMap* map, const void* base, uint64_t units, uint64_t heads,
                       uint64_t pages, uint64_t head_bytes, uint64_t page_bytes, uint32_t box);

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
// What the append reads and writes; sizes are the launcher's to fill in.
struct AppendArgs {
  RowsArg q, k, v, q_out;
  const float *cos_tab, *sin_tab;  // [angles][32]
  int angles;
  const int32_t *slots, *cu, *lens;
  PoolArg kc, vc;  // strides in elements (16-bit pools) or bytes (4-bit)
  int tokens, batch, H, Hkv, pages, shift;
  int parts;  // warps a token
  uint32_t* err;
};
int launch_paged_append(const PagedDims& d, const DevCtx& ctx, AppendArgs args, bool rotate,
                        bool four, cudaStream_t stream);
int launch_paged_load4(const PagedDims& d, const DevCtx& ctx, const PoolArg& kc, const PoolArg& vc,
                       const int32_t* slots, const RowsArg& k, const RowsArg& v,
                       cudaStream_t stream);
size_t paged_workspace_bytes(const PagedDims& d);
int launch_paged_fwd(const PagedDims& d, const DevCtx& ctx, const RowsArg& q, const PoolArg& kc,
                     const PoolArg& vc, const int32_t* table, const int32_t* cu,
                     const int32_t* lens, void* ws, bool four, const RowsArg& o, float* lse,
                     cudaStream_t stream);

}  // namespace css
