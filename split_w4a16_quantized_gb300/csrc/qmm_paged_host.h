// Launchers of the paged-cache calls (arguments checked by qmm_host.cpp).
#pragma once

#include <cstddef>
#include <cstdint>

#include "qmm.h"

namespace qmm {

// Paged cache (qmm_paged.cu): append with rotation, and the accepted path's
// walk and moves for the n caches of one launch.  axes: nullable; positions are
// then [axes->axes][N].
constexpr int kMaxTree = 256;          // drafted tokens per sequence
constexpr int kMaxAcceptCaches = 64;   // caches per qmm_tree_accept launch
int launch_kv_append(const qmm_kv_cache& c, const void* q, const void* k, const void* v,
                     void* q_out, int N, int Hq, int64_t q_stride, int64_t k_stride,
                     int64_t v_stride, int64_t q_out_stride, const int* cu, const int* positions,
                     const qmm_rope* rope, const qmm_rope_axes* axes, void* stream);
// outputs: whether this launch writes path, count, next and new_lens
int launch_tree_accept(const qmm_kv_cache* caches, int n, const int* tokens, const int* targets,
                       const int* parents, const int* cu, int N, int T, int* path, int* count,
                       int* next, int* new_lens, bool outputs, void* stream);
// Eviction (qmm_evict.cu) from the n caches of one launch, layers first .. first + n - 1
// of the weights and of kept.
constexpr int kMaxEvictCaches = 64;
int launch_kv_evict(const qmm_kv_cache* caches, int n, int first, const float* mass,
                    float* mass_out, int64_t layer_stride, int64_t row_stride, int keep, int sinks,
                    int recent, int* kept, int* new_lens, int num_sms, void* stream);
// Tree attention (qmm_tree_attention.cu).  lse: nullable, [B][T][Hq], log2 of each row's
// sum of 2^(score log2(e)).
size_t tree_attention_workspace(int D, int rows, int num_sms);
int launch_tree_attention(const qmm_kv_cache& c, const void* q, int64_t q_stride, void* O, int N,
                          int T, int Hq, const int* cu, const int* parents, float scale,
                          float* ws, int num_sms, void* stream, float* lse = nullptr);
// Attention that adds up the weights (qmm_scored_attention.cu).
size_t scored_attention_workspace(const qmm_kv_cache& c, int T, int Hq, int num_sms);
int launch_scored_attention(const qmm_kv_cache& c, const void* q, int64_t q_stride, void* O, int N,
                            int T, int Hq, const int* cu, float scale, float* mass,
                            int64_t mass_stride, float decay, float* ws, int num_sms,
                            void* stream);
// The weights of more than 8 rows per KV head, once each row's lse is there (qmm_mass_tc.cu).
int launch_mass_tc(const qmm_kv_cache& c, const void* q, int64_t q_stride, int N, int T, int Hq,
                   const int* cu, float scale, const float* lse, float* mass, int64_t mass_stride,
                   float decay, int num_sms, void* stream);
// Tree attention with shared prefixes (qmm_prefix_attention.cu); rows: N * Hq.
size_t prefix_attention_workspace(int D, int64_t rows, int B, int num_sms);
int launch_prefix_attention(const qmm_kv_cache& c, const qmm_prefix& pre, const void* q,
                            int64_t q_stride, void* O, int N, int T, int Hq, const int* cu,
                            const int* parents, float scale, float* ws, int num_sms,
                            void* stream);

}  // namespace qmm
