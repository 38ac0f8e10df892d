// chunk_api.cu — the C entries of pkv_chunk.h: host-side validation and the
// launches.  Nothing here allocates device memory or synchronises a stream.
#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include "chunk_internal.h"

namespace {

pkv_status fail(pkv_status s, const char* fmt, ...) {
  char msg[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof(msg), fmt, ap);
  va_end(ap);
  return pkv::record_error(s, msg);
}

pkv_status cuda_fail(cudaError_t e, const char* what) {
  return fail(PKV_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }

bool element_type(pkv_kv_dtype d) { return d == PKV_KV_F16 || d == PKV_KV_BF16 || d == PKV_KV_F32; }

int element_bytes(pkv_kv_dtype d) { return d == PKV_KV_F32 ? 4 : 2; }

// A token array of `heads` heads: its pointer and token stride.
pkv_status check_tokens(const char* name, const void* p, long long stride, int heads, pkv_kv_dtype d) {
  if (!p) return fail(PKV_ERR_INVALID_ARG, "null %s", name);
  if (!aligned(p, 16)) return fail(PKV_ERR_INVALID_ARG, "%s not 16-byte aligned", name);
  if (stride < static_cast<long long>(heads) * PKV_HEAD_DIM || stride >= (1ll << 31))
    return fail(PKV_ERR_INVALID_ARG, "%s_stride %lld below %lld, or 2^31 or more", name, stride,
                static_cast<long long>(heads) * PKV_HEAD_DIM);
  if (stride * element_bytes(d) % 16)
    return fail(PKV_ERR_INVALID_ARG, "%s_stride %lld not a multiple of 16 bytes", name, stride);
  return PKV_OK;
}

pkv_status check_rows(int num_rows, int total_tokens, const int32_t* cu, const int32_t* seq_lens,
                      const int32_t* bt, int bt_stride) {
  if (num_rows < 0 || total_tokens < 0)
    return fail(PKV_ERR_INVALID_ARG, "num_rows or total_tokens < 0");
  if (num_rows > PKV_MAX_ROWS)
    return fail(PKV_ERR_UNSUPPORTED, "num_rows %d > %d", num_rows, PKV_MAX_ROWS);
  if (total_tokens > PKV_MAX_CHUNK_TOKENS)
    return fail(PKV_ERR_UNSUPPORTED, "total_tokens %d > %d", total_tokens, PKV_MAX_CHUNK_TOKENS);
  if (bt_stride < 1 || bt_stride >= (1 << 27)) return fail(PKV_ERR_INVALID_ARG, "bt_stride outside [1, 2^27)");
  if (num_rows > 0 && (!cu || !seq_lens || !bt))
    return fail(PKV_ERR_INVALID_ARG, "null cu_seqlens, seq_lens or block table");
  if (!aligned(cu, 4) || !aligned(seq_lens, 4) || !aligned(bt, 4))
    return fail(PKV_ERR_INVALID_ARG, "cu_seqlens / seq_lens / block table not 4-byte aligned");
  return PKV_OK;
}

pkv_status check_group(int n_q, int n_kv) {
  if (n_q <= 0) return fail(PKV_ERR_INVALID_ARG, "n_q_heads must be positive");
  if (n_q % n_kv) return fail(PKV_ERR_INVALID_ARG, "n_q_heads %% n_kv_heads != 0");
  const int g = n_q / n_kv;
  if (g != 1 && g != 2 && g != 4) return fail(PKV_ERR_UNSUPPORTED, "GQA group %d not in {1,2,4}", g);
  return PKV_OK;
}

pkv_status check_scores(const pkv_scores* sc) {
  if (!sc) return fail(PKV_ERR_INVALID_ARG, "null scores");
  if (!std::isfinite(sc->scale)) return fail(PKV_ERR_INVALID_ARG, "scale is not finite");
  if (!(sc->softcap >= 0.0f) || !std::isfinite(sc->softcap))
    return fail(PKV_ERR_INVALID_ARG, "softcap below 0 or not finite");
  if (sc->softcap > 0.0f && (sc->softcap < 1e-30f || sc->softcap > 1e30f || !std::isfinite(sc->scale / sc->softcap)))
    return fail(PKV_ERR_INVALID_ARG, "softcap outside 1e-30 .. 1e30, or scale / softcap not finite");
  if (!aligned(sc->slopes, 4) || !aligned(sc->prefix_lens, 4))
    return fail(PKV_ERR_INVALID_ARG, "slopes / prefix_lens not 4-byte aligned");
  return PKV_OK;
}

// The type a pool's chunk attention takes its queries in.
pkv_status check_q_type(int pool_dtype, pkv_kv_dtype q_dtype) {
  if (pool_dtype == PKV_KV_F32)
    return fail(PKV_ERR_UNSUPPORTED, "chunk attention takes f16, bf16 and q8_0 pools");
  const pkv_kv_dtype want = pool_dtype == PKV_KV_BF16 ? PKV_KV_BF16 : PKV_KV_F16;
  if (q_dtype != want)
    return fail(PKV_ERR_UNSUPPORTED, "q_dtype %d: this pool takes %s queries", static_cast<int>(q_dtype),
                want == PKV_KV_BF16 ? "bf16" : "f16");
  return PKV_OK;
}

pkv::ChunkRows rows_of(const int32_t* cu, const int32_t* seq_lens, const int32_t* bt, int bt_stride,
                       int num_rows, int total_tokens) {
  return pkv::ChunkRows{cu, seq_lens, bt, bt_stride, num_rows, total_tokens};
}

pkv_status default_chunks(int* chunks) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceGetAttribute");
  *chunks = sms;
  return PKV_OK;
}

constexpr int kMaxChunks = 4096;

}  // namespace

extern "C" {

pkv_status kv_rope_append(const pkv_pool* pool, int layer, const void* q, long long q_stride,
                          const void* k, long long k_stride, const void* v, long long v_stride,
                          pkv_kv_dtype in_dtype, void* q_out, pkv_kv_dtype q_dtype,
                          const int32_t* positions, int num_axes, const int* sections,
                          const float* inv_freq, int rot_dim, int interleaved,
                          const int32_t* cu_seqlens, int total_tokens, const int32_t* block_table,
                          int bt_stride, const int32_t* seq_lens, int num_rows, int n_q_heads,
                          void* stream) {
  pkv::RopeArgs a;
  pkv_status s = pkv::pool_layer_view(pool, layer, &a.pool);
  if (s) return s;
  if ((s = check_rows(num_rows, total_tokens, cu_seqlens, seq_lens, block_table, bt_stride))) return s;
  if (!element_type(in_dtype) || !element_type(q_dtype))
    return fail(PKV_ERR_UNSUPPORTED, "in_dtype and q_dtype must be f16, bf16 or f32");
  if (n_q_heads < 0 || n_q_heads > (1 << 16)) return fail(PKV_ERR_INVALID_ARG, "n_q_heads outside [0, 65536]");
  if (rot_dim < 16 || rot_dim > PKV_HEAD_DIM || rot_dim % 16)
    return fail(PKV_ERR_UNSUPPORTED, "rot_dim %d not a multiple of 16 in [16, 128]", rot_dim);
  if (num_axes < 1 || num_axes > PKV_MAX_ROPE_AXES)
    return fail(PKV_ERR_UNSUPPORTED, "num_axes %d outside [1, %d]", num_axes, PKV_MAX_ROPE_AXES);
  if (!sections) return fail(PKV_ERR_INVALID_ARG, "null sections");
  int end = 0;
  for (int x = 0; x < PKV_MAX_ROPE_AXES; ++x) {
    if (x < num_axes) {
      if (sections[x] < 1 || sections[x] > PKV_HEAD_DIM)
        return fail(PKV_ERR_INVALID_ARG, "sections[%d] = %d outside [1, 128]", x, sections[x]);
      end += sections[x];
    }
    a.axis_end[x] = end;
  }
  if (end != rot_dim / 2)
    return fail(PKV_ERR_INVALID_ARG, "sections sum to %d, not rot_dim / 2 = %d", end, rot_dim / 2);
  if (num_rows == 0 || total_tokens == 0) return PKV_OK;
  if (n_q_heads > 0) {
    if ((s = check_tokens("q", q, q_stride, n_q_heads, in_dtype))) return s;
    if (!q_out) return fail(PKV_ERR_INVALID_ARG, "null q_out");
    if (!aligned(q_out, 16)) return fail(PKV_ERR_INVALID_ARG, "q_out not 16-byte aligned");
    if (q == q_out && (in_dtype != q_dtype || q_stride != static_cast<long long>(n_q_heads) * PKV_HEAD_DIM))
      return fail(PKV_ERR_INVALID_ARG, "q_out is q, but of another type or stride");
  }
  if ((s = check_tokens("k", k, k_stride, a.pool.n_kv, in_dtype))) return s;
  if ((s = check_tokens("v", v, v_stride, a.pool.n_kv, in_dtype))) return s;
  if (!positions || !inv_freq) return fail(PKV_ERR_INVALID_ARG, "null positions or inv_freq");
  if (!aligned(positions, 4) || !aligned(inv_freq, 4))
    return fail(PKV_ERR_INVALID_ARG, "positions / inv_freq not 4-byte aligned");
  a.rows = rows_of(cu_seqlens, seq_lens, block_table, bt_stride, num_rows, total_tokens);
  a.q = static_cast<const uint8_t*>(q);
  a.k = static_cast<const uint8_t*>(k);
  a.v = static_cast<const uint8_t*>(v);
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_out = static_cast<uint8_t*>(q_out);
  a.positions = positions;
  a.inv_freq = inv_freq;
  a.in_dtype = in_dtype;
  a.q_dtype = q_dtype;
  a.n_q = n_q_heads;
  a.half = rot_dim / 2;
  a.interleaved = interleaved != 0;
  const cudaError_t e = pkv::launch_rope_append(a, as_stream(stream));
  if (e != cudaSuccess) return cuda_fail(e, "kv_rope_append launch");
  return PKV_OK;
}

size_t paged_chunk_workspace_bytes(const pkv_pool* pool, int n_q_heads, int num_chunks) {
  const int n_kv = pkv::pool_kv_heads(pool);
  if (n_kv <= 0 || check_group(n_q_heads, n_kv) || num_chunks < 1 || num_chunks > kMaxChunks) return 0;
  return pkv::chunk_attention_workspace(n_q_heads, n_kv, num_chunks);
}

size_t paged_attention_mass_workspace_bytes(int num_chunks) {
  return num_chunks < 1 || num_chunks > kMaxChunks ? 0 : pkv::attention_mass_workspace(num_chunks);
}

pkv_status paged_chunk_default_chunks(const pkv_pool* pool, int n_q_heads, int* chunks) {
  if (!pool || !chunks) return fail(PKV_ERR_INVALID_ARG, "null pool or output pointer");
  const pkv_status s = check_group(n_q_heads, pkv::pool_kv_heads(pool));
  if (s) return s;
  return default_chunks(chunks);
}

pkv_status paged_chunk_attention(const pkv_pool* pool, int layer, const void* q, long long q_stride,
                                 pkv_kv_dtype q_dtype, const int32_t* cu_seqlens, int total_tokens,
                                 const int32_t* block_table, int bt_stride,
                                 const int32_t* seq_lens, int num_rows, int n_q_heads,
                                 const pkv_scores* scores, void* out, float* lse, void* workspace,
                                 size_t workspace_bytes, int num_chunks, void* stream) {
  pkv::ChunkAttnArgs a;
  pkv_status s = pkv::pool_layer_view(pool, layer, &a.pool);
  if (s) return s;
  if ((s = check_group(n_q_heads, a.pool.n_kv))) return s;
  if ((s = check_q_type(a.pool.dtype, q_dtype))) return s;
  if ((s = check_rows(num_rows, total_tokens, cu_seqlens, seq_lens, block_table, bt_stride))) return s;
  if ((s = check_scores(scores))) return s;
  if (num_chunks < 0) return fail(PKV_ERR_INVALID_ARG, "num_chunks < 0");
  if (num_chunks > kMaxChunks) return fail(PKV_ERR_UNSUPPORTED, "num_chunks > %d", kMaxChunks);
  if (num_rows == 0 || total_tokens == 0) return PKV_OK;
  if ((s = check_tokens("q", q, q_stride, n_q_heads, q_dtype))) return s;
  if (!out) return fail(PKV_ERR_INVALID_ARG, "null out");
  if (!aligned(out, 16) || !aligned(lse, 4)) return fail(PKV_ERR_INVALID_ARG, "out or lse not aligned");
  if (num_chunks == 0 && (s = default_chunks(&num_chunks))) return s;
  const size_t need = pkv::chunk_attention_workspace(n_q_heads, a.pool.n_kv, num_chunks);
  if (!workspace || workspace_bytes < need)
    return fail(PKV_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
  if (!aligned(workspace, 256)) return fail(PKV_ERR_INVALID_ARG, "workspace not 256-byte aligned");
  // a row that is computed again reads its query after others are written
  if (out == q) return fail(PKV_ERR_INVALID_ARG, "out must not be q");
  a.rows = rows_of(cu_seqlens, seq_lens, block_table, bt_stride, num_rows, total_tokens);
  a.q = static_cast<const uint8_t*>(q);
  a.q_stride = q_stride;
  a.n_q = n_q_heads;
  a.sc = pkv::ScoreArgs{scores->scale, scores->softcap, scores->slopes, scores->prefix_lens};
  a.out = static_cast<uint8_t*>(out);
  a.lse = lse;
  a.workspace = static_cast<uint8_t*>(workspace);
  a.chunks = num_chunks;
  const pkv::TileMaps* maps = nullptr;
  if ((s = pkv::pool_layer_maps(pool, layer, &maps))) return s;
  const cudaError_t e = pkv::launch_chunk_attention(a, *maps, as_stream(stream));
  if (e != cudaSuccess) return cuda_fail(e, "chunk attention launch");
  return PKV_OK;
}

pkv_status paged_attention_mass(const pkv_pool* pool, int layer, const void* q, long long q_stride,
                                pkv_kv_dtype q_dtype, const float* lse, const int32_t* cu_seqlens,
                                int total_tokens, const int32_t* block_table, int bt_stride,
                                const int32_t* seq_lens, int num_rows, int n_q_heads,
                                const pkv_scores* scores, int last_queries, const float* mass_in,
                                float* mass_out, int mass_stride, void* workspace,
                                size_t workspace_bytes, int num_chunks, void* stream) {
  pkv::MassArgs a;
  pkv_status s = pkv::pool_layer_view(pool, layer, &a.pool);
  if (s) return s;
  if ((s = check_group(n_q_heads, a.pool.n_kv))) return s;
  if ((s = check_q_type(a.pool.dtype, q_dtype))) return s;
  if ((s = check_rows(num_rows, total_tokens, cu_seqlens, seq_lens, block_table, bt_stride))) return s;
  if ((s = check_scores(scores))) return s;
  if (last_queries < 0) return fail(PKV_ERR_INVALID_ARG, "last_queries < 0");
  if (mass_stride < 1) return fail(PKV_ERR_INVALID_ARG, "mass_stride < 1");
  if (num_chunks < 0) return fail(PKV_ERR_INVALID_ARG, "num_chunks < 0");
  if (num_chunks > kMaxChunks) return fail(PKV_ERR_UNSUPPORTED, "num_chunks > %d", kMaxChunks);
  if (num_rows == 0 || total_tokens == 0) return PKV_OK;
  if ((s = check_tokens("q", q, q_stride, n_q_heads, q_dtype))) return s;
  if (!lse) return fail(PKV_ERR_INVALID_ARG, "null lse");
  if (!mass_out) return fail(PKV_ERR_INVALID_ARG, "null mass_out");
  if (!aligned(lse, 4) || !aligned(mass_in, 4) || !aligned(mass_out, 4))
    return fail(PKV_ERR_INVALID_ARG, "lse / mass not 4-byte aligned");
  a.rows = rows_of(cu_seqlens, seq_lens, block_table, bt_stride, num_rows, total_tokens);
  a.q = static_cast<const uint8_t*>(q);
  a.q_stride = q_stride;
  a.n_q = n_q_heads;
  a.sc = pkv::ScoreArgs{scores->scale, scores->softcap, scores->slopes, scores->prefix_lens};
  a.lse = lse;
  a.last_queries = last_queries;
  a.mass_in = mass_in;
  a.mass_out = mass_out;
  a.mass_stride = mass_stride;
  if (num_chunks == 0 && (s = default_chunks(&num_chunks))) return s;
  const size_t need = pkv::attention_mass_workspace(num_chunks);
  if (!workspace || workspace_bytes < need)
    return fail(PKV_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
  if (!aligned(workspace, 256)) return fail(PKV_ERR_INVALID_ARG, "workspace not 256-byte aligned");
  a.workspace = static_cast<uint8_t*>(workspace);
  a.chunks = num_chunks;
  const pkv::TileMaps* maps = nullptr;
  if ((s = pkv::pool_layer_maps(pool, layer, &maps))) return s;
  const cudaError_t e = pkv::launch_attention_mass(a, *maps, as_stream(stream));
  if (e != cudaSuccess) return cuda_fail(e, "attention mass launch");
  return PKV_OK;
}

pkv_status kv_evict(const pkv_pool* pool, int layer, const float* mass, int mass_stride,
                    const int32_t* block_table, int bt_stride, const int32_t* seq_lens,
                    int num_rows, const int32_t* keep_lens, int first, int recent,
                    const int32_t* dst_block_table, int dst_bt_stride, int32_t* keep_idx,
                    int keep_stride, float* dst_mass, int32_t* new_lens, void* stream) {
  pkv::EvictArgs a;
  pkv_status s = pkv::pool_layer_view(pool, layer, &a.pool);
  if (s) return s;
  if (num_rows < 0) return fail(PKV_ERR_INVALID_ARG, "num_rows < 0");
  if (num_rows > PKV_MAX_ROWS) return fail(PKV_ERR_UNSUPPORTED, "num_rows %d > %d", num_rows, PKV_MAX_ROWS);
  if (bt_stride < 1 || dst_bt_stride < 1 || bt_stride >= (1 << 27) || dst_bt_stride >= (1 << 27))
    return fail(PKV_ERR_INVALID_ARG, "bt_stride or dst_bt_stride outside [1, 2^27)");
  if (mass_stride < 1 || keep_stride < 1)
    return fail(PKV_ERR_INVALID_ARG, "mass_stride or keep_stride < 1");
  if (first < 0 || recent < 0) return fail(PKV_ERR_INVALID_ARG, "first or recent < 0");
  if (a.pool.n_kv > 65535) return fail(PKV_ERR_UNSUPPORTED, "n_kv_heads %d > 65535", a.pool.n_kv);
  if (num_rows == 0) return PKV_OK;
  if (!mass || !block_table || !seq_lens || !keep_lens || !dst_block_table || !keep_idx || !new_lens)
    return fail(PKV_ERR_INVALID_ARG, "null argument");
  if (!aligned(mass, 4) || !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(keep_lens, 4) ||
      !aligned(dst_block_table, 4) || !aligned(keep_idx, 4) || !aligned(dst_mass, 4) || !aligned(new_lens, 4))
    return fail(PKV_ERR_INVALID_ARG, "an argument is not 4-byte aligned");
  if (new_lens == seq_lens || new_lens == keep_lens)
    return fail(PKV_ERR_INVALID_ARG, "new_lens must be an array of its own");
  if (dst_mass == mass) return fail(PKV_ERR_INVALID_ARG, "dst_mass must not be mass");
  a.mass = mass;
  a.mass_stride = mass_stride;
  a.block_table = block_table;
  a.bt_stride = bt_stride;
  a.seq_lens = seq_lens;
  a.num_rows = num_rows;
  a.keep_lens = keep_lens;
  a.first = first;
  a.recent = recent;
  a.dst_block_table = dst_block_table;
  a.dst_bt_stride = dst_bt_stride;
  a.keep_idx = keep_idx;
  a.keep_stride = keep_stride;
  a.dst_mass = dst_mass;
  a.new_lens = new_lens;
  const cudaError_t e = pkv::launch_evict(a, as_stream(stream));
  if (e != cudaSuccess) return cuda_fail(e, "kv_evict launch");
  return PKV_OK;
}

}  // extern "C"
