/*
 * A plain C99 client of the FP8 layer and the mixture-of-experts layer (include/w4a4.h).
 *
 *   w4a4_fp8_client host
 *       prints the sizes of the descriptors and layouts and some size queries.
 *   w4a4_fp8_client run IN OUT
 *       reads T, d, f, E, k (int64), X [T][d], router [E][d], gate [E][f][d], up [E][f][d],
 *       down [E][d][f], Wo [d][d] (fp32) from IN; packs, runs the linear layer of Wo and the gated
 *       experts on the current HIP device, and writes both outputs [T][d] (fp32) to OUT.
 * Exit status 0 on success; any failing call prints its status name and exits 1.
 */
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <hip/hip_runtime_api.h>

#include "w4a4.h"

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
static void* read_to_device(FILE* f, int64_t n) {
    const size_t bytes = (size_t)n * sizeof(float);
    void* h = malloc(bytes);
    void* d = device(bytes);
    if (!h || fread(h, 1, bytes, f) != bytes) {
        fprintf(stderr, "short read\n");
        exit(1);
    }
    check_hip(hipMemcpy(d, h, bytes, hipMemcpyHostToDevice), "hipMemcpy");
    free(h);
    return d;
}
static w4a4_fp8_packed pack(const void* W, int64_t n_mat, int64_t d_in, int64_t d_out) {
    w4a4_fp8_packed p;
    size_t n = 0;
    void* blob;
    check(w4a4_fp8_packed_size(n_mat, d_in, d_out, &n), "w4a4_fp8_packed_size");
    blob = device(n);
    check(w4a4_fp8_pack_weights(W, W4A4_X_F32, n_mat, d_in, d_out, W4A4_FP8_SCALE_F32, blob, n, &p, NULL), "w4a4_fp8_pack_weights");
    return p;
}

static int host_mode(void) {
    size_t n = 0;
    printf("packed %zu\n", sizeof(w4a4_fp8_packed));
    printf("ws_layout %zu\n", sizeof(w4a4_fp8_ws_layout));
    printf("moe %zu\n", sizeof(w4a4_moe));
    printf("moe_ws_layout %zu\n", sizeof(w4a4_moe_ws_layout));
    check(w4a4_fp8_packed_size(3, 300, 200, &n), "w4a4_fp8_packed_size");
    printf("packed_size %zu\n", n);
    printf("packed_size_none %d\n", w4a4_fp8_packed_size(0, 300, 200, &n));
    return 0;
}

static int run_mode(const char* in, const char* out) {
    FILE* f = fopen(in, "rb");
    int64_t h[5];
    int64_t T, d, fw, E;
    size_t n = 0, bytes;
    w4a4_fp8_packed wo;
    w4a4_moe moe;
    void *X, *router, *Y, *ws;
    float* y;
    int i;
    if (!f || fread(h, sizeof(int64_t), 5, f) != 5) return 1;
    T = h[0], d = h[1], fw = h[2], E = h[3];
    X = read_to_device(f, T * d);
    router = read_to_device(f, E * d);
    memset(&moe, 0, sizeof moe);
    moe.gate = pack(read_to_device(f, E * fw * d), E, d, fw);
    moe.up = pack(read_to_device(f, E * fw * d), E, d, fw);
    moe.down = pack(read_to_device(f, E * d * fw), E, fw, d);
    wo = pack(read_to_device(f, d * d), 1, d, d);
    fclose(f);
    moe.router = router;
    moe.router_dtype = W4A4_X_F32;
    moe.top_k = (int32_t)h[4];
    moe.renormalize = 1;
    moe.activation = W4A4_MOE_SILU_GATED;
    bytes = (size_t)(T * d) * sizeof(float);
    Y = device(bytes);
    y = (float*)malloc(bytes);
    f = fopen(out, "wb");
    if (!y || !f) return 1;
    for (i = 0; i < 2; ++i) {
        if (i == 0) check(w4a4_fp8_workspace_size(T, &wo, &n), "w4a4_fp8_workspace_size");
        else check(w4a4_moe_workspace_size(T, &moe, &n), "w4a4_moe_workspace_size");
        ws = device(n);
        if (i == 0) check(w4a4_fp8_linear(X, W4A4_X_F32, T, &wo, Y, W4A4_Y_F32, ws, n, NULL), "w4a4_fp8_linear");
        else check(w4a4_moe_forward(X, W4A4_X_F32, T, &moe, Y, W4A4_Y_F32, ws, n, NULL), "w4a4_moe_forward");
        check_hip(hipDeviceSynchronize(), "hipDeviceSynchronize");
        check_hip(hipMemcpy(y, Y, bytes, hipMemcpyDeviceToHost), "hipMemcpy");
        if (fwrite(y, 1, bytes, f) != bytes) return 1;
    }
    return fclose(f);
}

int main(int argc, char** argv) {
    if (argc == 2 && strcmp(argv[1], "host") == 0) return host_mode();
    if (argc == 4 && strcmp(argv[1], "run") == 0) return run_mode(argv[2], argv[3]);
    fprintf(stderr, "usage: %s host | run IN OUT\n", argv[0]);
    return 2;
}
