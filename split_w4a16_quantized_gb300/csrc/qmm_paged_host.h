// Launchers of the paged-cache calls (arguments checked by qmm_host.cpp).
#pragma once

#include <cstddef>
#include <cstdint>

#include "qmm.h"

namespace qmm {

// Paged cache (qmm_paged.cu): append with rotation, and the accepted path's
// walk and moves for the n caches of one launch.
constexpr int kMaxTree = 256;          // drafted tokens per sequence
constexpr int kMaxAcceptCaches = 64;   // caches per qmm_tree_accept launch
int launch_kv_append(const qmm_kv_cache& c, const void* q, const void* k, const void* v,
                     void* q_out, int N, int Hq, int64_t q_stride, int64_t k_stride,
                     int64_t v_stride, int64_t q_out_stride, const int* cu, const int* positions,
                     const qmm_rope* rope, void* stream);
// outputs: whether this launch writes path, count, next and new_lens
int launch_tree_accept(const qmm_kv_cache* caches, int n, const int* tokens, const int* targets,
                       const int* parents, const int* cu, int N, int T, int* path, int* count,
                       int* next, int* new_lens, bool outputs, void* stream);
// Tree attention (qmm_tree_attention.cu).
size_t tree_attention_workspace(int D, int rows, int num_sms);
int launch_tree_attention(const qmm_kv_cache& c, const void* q, int64_t q_stride, void* O, int N,
                          int T, int Hq, const int* cu, const int* parents, float scale,
                          float* ws, int num_sms, void* stream);

}  // namespace qmm
