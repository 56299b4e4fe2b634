// e4m3_plan_dump.cu -- prints which kernel the e4m3 products would choose:
// reads lines "rows inner outer experts", writes "many" or "few <tokens a
// tile> <blocks that split K>" for each.  Linked against libqgemv.so, run on
// the GPU whose cluster counts the choice asks for.
#include <cstdio>

#include "gemm_e4m3_tc.cuh"

int main() {
    int M, I, O, E;
    while (scanf("%d %d %d %d", &M, &I, &O, &E) == 4) {
        const qg::e8::FewPlan few = qg::e8::plan_few(M, I, O, E);
        const qg::e8::ManyPlan many = qg::e8::plan_many(M, I, O, E);
        if (many.cost < few.cost) printf("many\n");
        else printf("few %d %d\n", few.bt, few.cluster);
    }
    return 0;
}
