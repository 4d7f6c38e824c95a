/*
 * A plain C99 client of the INT8 layer, the 4-bit key/value cache and attention over it (include/w4a4.h).
 *
 *   w4a4_kv_client host
 *       prints the sizes of the descriptors and some size queries.
 *   w4a4_kv_client run IN OUT
 *       reads T, d, Hq, H, D (int64), X [T][d], W [(Hq + 2 H) D][d] (fp32) from IN; one sequence of T
 *       tokens: projects X to queries, keys and values in INT8, writes keys and values into a
 *       cache of pages in descending order, attends (causal), reads the cache back, and writes
 *       the projections (fp32), the attention's outputs (bf16) and the keys and values (fp32) to OUT.
 * Exit status 0 on success; any failing call prints its status name and exits 1.
 */
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include <hip/hip_runtime_api.h>

#include "w4a4.h"

enum { PAGE = 16 };

static void check(int st, const char* what) {
    if (st != W4A4_OK) {
        fprintf(stderr, "%s failed: %s\n", what, w4a4_status_string(st));
        exit(1);
    }
}
static void check_hip(hipError_t e, const char* what) {
    if (e != hipSuccess) {
        fprintf(stderr, "%s failed: %s\n", what, hipGetErrorString(e));
        exit(1);
    }
}
static void* device(size_t n) {
    void* d = NULL;
    check_hip(hipMalloc(&d, n > 0 ? n : 1), "hipMalloc");
    return d;
}
static void* to_device(const void* h, size_t bytes) {
    void* d = device(bytes);
    check_hip(hipMemcpy(d, h, bytes, hipMemcpyHostToDevice), "hipMemcpy");
    return d;
}
static void* read_to_device(FILE* f, int64_t n) {
    const size_t bytes = (size_t)n * sizeof(float);
    void* h = malloc(bytes);
    void* d;
    if (!h || fread(h, 1, bytes, f) != bytes) {
        fprintf(stderr, "short read\n");
        exit(1);
    }
    d = to_device(h, bytes);
    free(h);
    return d;
}
static void write_out(FILE* f, const void* d, size_t bytes) {
    void* h = malloc(bytes);
    if (!h) exit(1);
    check_hip(hipMemcpy(h, d, bytes, hipMemcpyDeviceToHost), "hipMemcpy");
    if (fwrite(h, 1, bytes, f) != bytes) exit(1);
    free(h);
}

static int host_mode(void) {
    size_t n = 0;
    printf("int8_packed %zu\n", sizeof(w4a4_int8_packed));
    printf("int8_ws_layout %zu\n", sizeof(w4a4_int8_ws_layout));
    printf("cache %zu\n", sizeof(w4a4_kv_cache));
    printf("batch %zu\n", sizeof(w4a4_kv_batch));
    printf("rows %zu\n", sizeof(w4a4_kv_rows));
    check(w4a4_int8_packed_size(300, 200, &n), "w4a4_int8_packed_size");
    printf("int8_packed_size %zu\n", n);
    check(w4a4_kv_cache_size(7, 32, 3, 72, &n), "w4a4_kv_cache_size");
    printf("cache_size %zu\n", n);
    printf("cache_size_none %d\n", w4a4_kv_cache_size(7, 20, 3, 72, &n));
    return 0;
}

static int run_mode(const char* in, const char* out) {
    FILE* f = fopen(in, "rb");
    int64_t h[5], T, d, Hq, H, D, wide, n_pages, i;
    int32_t* table;
    int32_t start[2], len[1];
    size_t n = 0, kv_bytes;
    w4a4_int8_packed w;
    w4a4_kv_cache cache;
    w4a4_kv_batch batch;
    w4a4_kv_rows q, k, v;
    void *X, *W, *P, *O, *K, *V, *ws;
    if (!f || fread(h, sizeof(int64_t), 5, f) != 5) return 1;
    T = h[0], d = h[1], Hq = h[2], H = h[3], D = h[4];
    wide = (Hq + 2 * H) * D;
    X = read_to_device(f, T * d);
    W = read_to_device(f, wide * d);
    fclose(f);

    check(w4a4_int8_packed_size(d, wide, &n), "w4a4_int8_packed_size");
    check(w4a4_int8_pack_weights(W, W4A4_X_F32, d, wide, device(n), n, &w, NULL), "w4a4_int8_pack_weights");
    check(w4a4_int8_workspace_size(T, &w, &n), "w4a4_int8_workspace_size");
    P = device((size_t)(T * wide) * sizeof(float));
    check(w4a4_int8_linear(X, W4A4_X_F32, T, &w, P, W4A4_Y_F32, device(n), n, NULL), "w4a4_int8_linear");

    n_pages = (T + PAGE - 1) / PAGE;
    table = (int32_t*)malloc((size_t)n_pages * sizeof(int32_t));
    if (!table) return 1;
    for (i = 0; i < n_pages; ++i) table[i] = (int32_t)(n_pages - 1 - i);
    start[0] = 0, start[1] = (int32_t)T, len[0] = (int32_t)T;
    check(w4a4_kv_cache_size(n_pages, PAGE, (int32_t)H, (int32_t)D, &n), "w4a4_kv_cache_size");
    check(w4a4_kv_cache_describe(n_pages, PAGE, (int32_t)H, (int32_t)D, device(n), n, &cache), "w4a4_kv_cache_describe");
    batch.n_seqs = 1, batch.max_rows = T, batch.max_pages = n_pages;
    batch.q_start = (const int32_t*)to_device(start, sizeof start);
    batch.lens = (const int32_t*)to_device(len, sizeof len);
    batch.pages = (const int32_t*)to_device(table, (size_t)n_pages * sizeof(int32_t));
    free(table);
    /* queries, keys and values are slices of the projections' rows */
    q.data = P, q.row_stride = wide, q.head_stride = D, q.dtype = W4A4_X_F32, q.reserved = 0;
    k = q, v = q;
    k.data = (const float*)P + Hq * D;
    v.data = (const float*)P + (Hq + H) * D;
    check(w4a4_kv_append(&k, &v, T, &batch, &cache, NULL), "w4a4_kv_append");
    check(w4a4_kv_attention_workspace_size(T, &batch, &cache, (int32_t)Hq, &n), "w4a4_kv_attention_workspace_size");
    ws = device(n);
    O = device((size_t)(T * Hq * D) * sizeof(uint16_t));
    check(w4a4_kv_attention(&q, T, &batch, &cache, (int32_t)Hq, 0.125f, 1, 0, (uint16_t*)O, ws, n, NULL), "w4a4_kv_attention");
    kv_bytes = (size_t)(T * H * D) * sizeof(float);
    K = device(kv_bytes);
    V = device(kv_bytes);
    check(w4a4_kv_read(T, &batch, &cache, K, V, W4A4_Y_F32, NULL), "w4a4_kv_read");
    check_hip(hipDeviceSynchronize(), "hipDeviceSynchronize");

    f = fopen(out, "wb");
    if (!f) return 1;
    write_out(f, P, (size_t)(T * wide) * sizeof(float));
    write_out(f, O, (size_t)(T * Hq * D) * sizeof(uint16_t));
    write_out(f, K, kv_bytes);
    write_out(f, V, kv_bytes);
    return fclose(f);
}

int main(int argc, char** argv) {
    if (argc == 2 && argv[1][0] == 'h') return host_mode();
    if (argc == 4 && argv[1][0] == 'r') return run_mode(argv[2], argv[3]);
    fprintf(stderr, "usage: %s host | run IN OUT\n", argv[0]);
    return 2;
}
