// Host build of the draft tree's steps (causal_attention_sdpa_b200/csrc/paging.h) as the kernels take
// them, arrays in place of the shuffles of a warp, for the CPU tests.
#include "paging.h"

using namespace gpt_attn;

extern "C" {
// Ancestors and depth of all kMaxNodes nodes.
void tree_all(int N, const int* parents, unsigned long long* anc, int* depth) {
    TreeNode x[kMaxNodes], next[kMaxNodes];
    for (int n = 0; n < kMaxNodes; ++n) x[n] = tree_node(n, n < N ? parents[n] : -1);
    for (int step = 1; step < N; step *= 2) {
        for (int n = 0; n < kMaxNodes; ++n) next[n] = tree_step(x[n], x[x[n].up < 0 ? 0 : x[n].up]);
        for (int n = 0; n < kMaxNodes; ++n) x[n] = next[n];
    }
    for (int n = 0; n < kMaxNodes; ++n) {
        anc[n] = x[n].anc;
        depth[n] = -1;
        for (unsigned long long a = x[n].anc; a; a &= a - 1) ++depth[n];
    }
}
int tree_pool_row(int entry, int in_page, int page, int n_pages, int Hkv, int h) {
    return pool_row(entry, in_page, fast_div(page), n_pages, Hkv, h);
}
}
